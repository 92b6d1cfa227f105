"""Cases that measure the rotary and cache operators of the Lighthouse library.

A user's path next to the layer: rotary positions on Q and K before it and
their gradient behind it (``lh.rotary``, ``lh.rotary_bwd``); and, to answer
with the trained model, a paged key-value cache that is filled
(``lh.cache_append``), read by the attention of one new token
(``lh.decode``) and kept short by accumulated attention weight (``lh.evict``).

``run`` computes each operator in plain torch operations when ``own`` is
false and through the library when it is true; ``exact`` gives the same
outputs from the definitions in 64 bits.
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"bf16": 2, "f32": 4}


# --- cases ---------------------------------------------------------------------


def listed():
    return [
        # Q and K of the layer at its 98,304-token benchmark shape, on their way into lh.forward
        {"name": "rotary_98k", "op": "rotary", "dtype": "bf16", "B": 1, "Hq": 16, "Hk": 16, "N": 98304,
         "d": 64, "rot": 64, "layout": "half", "scaling": "none", "base": 10000.0, "transpose": False,
         "rows": "heads", "packed": False, "start": 0},
        # the extreme length: far positions, frequencies scaled for the long context, read as the
        # projection leaves them (token-major)
        {"name": "rotary_512k_scaled", "op": "rotary", "dtype": "bf16", "B": 1, "Hq": 16, "Hk": 16, "N": 524288,
         "d": 64, "rot": 64, "layout": "half", "scaling": "bands", "base": 500000.0, "transpose": False,
         "rows": "tokens", "packed": False, "start": 0},
        # gradients behind lh.backward: packed documents of odd lengths, half of the head rotated
        {"name": "rotary_grad_8k_f32", "op": "rotary", "dtype": "f32", "B": 2, "Hq": 8, "Hk": 8, "N": 8191,
         "d": 64, "rot": 32, "layout": "interleaved", "scaling": "none", "base": 10000.0, "transpose": True,
         "rows": "heads", "packed": True, "start": 0},
        # gradients at head dimension 128 with fewer key heads, linear scaling, a continued sequence
        {"name": "rotary_grad_d128", "op": "rotary", "dtype": "bf16", "B": 1, "Hq": 8, "Hk": 2, "N": 98304,
         "d": 128, "rot": 128, "layout": "half", "scaling": "linear", "base": 10000.0, "transpose": True,
         "rows": "heads", "packed": False, "start": 4096},
        # one decoding step of a batch: the smallest calls, where latency counts
        {"name": "append_step", "op": "append", "dtype": "bf16", "B": 16, "Hq": 16, "Hk": 16, "T": 1, "d": 64,
         "page": 64, "length": 8192, "ragged": False, "layout": "half"},
        # prompts of unequal lengths written at once, padded to the longest
        {"name": "append_prompts", "op": "append", "dtype": "bf16", "B": 4, "Hq": 16, "Hk": 4, "T": 8192,
         "d": 128, "page": 64, "length": 8192, "ragged": True, "layout": "half"},
        # one short sequence, its pages ending inside a tile
        {"name": "decode_short", "op": "decode", "dtype": "bf16", "B": 1, "Hq": 16, "Hk": 2, "length": 37,
         "d": 64, "page": 16, "ragged": False, "weights": False},
        # one sequence at the benchmark's length, as many key heads as query heads
        {"name": "decode_98k", "op": "decode", "dtype": "bf16", "B": 1, "Hq": 16, "Hk": 16, "length": 98304,
         "d": 64, "page": 64, "ragged": False, "weights": False},
        # a serving batch of unequal lengths (an empty one among them), shared key heads
        {"name": "decode_batch", "op": "decode", "dtype": "bf16", "B": 64, "Hq": 16, "Hk": 4, "length": 16384,
         "d": 128, "page": 64, "ragged": True, "weights": False},
        # a step that also adds its probabilities to the cache's weights, in 32 bits
        {"name": "decode_weights_f32", "op": "decode", "dtype": "f32", "B": 2, "Hq": 16, "Hk": 8, "length": 8191,
         "d": 64, "page": 32, "ragged": False, "weights": True},
        # a long prompt's cache cut to half
        {"name": "evict_98k", "op": "evict", "dtype": "bf16", "B": 1, "Hk": 16, "d": 64, "page": 64,
         "length": 98304, "budget": 49152, "recent": 1024, "ragged": False, "positions": False},
        # the regular cut of a batch's caches after some steps of decoding
        {"name": "evict_step", "op": "evict", "dtype": "bf16", "B": 8, "Hk": 8, "d": 128, "page": 32,
         "length": 2111, "budget": 2048, "recent": 64, "ragged": True, "positions": True},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rotary", "rotary", "append", "decode", "decode", "evict"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    d = rng.choice([64, 128])
    Hk = rng.choice([1, 2, 4, 8, 16])
    es = SIZE[dtype]
    if op == "rotary":
        Hq = Hk * rng.choice([1, 1, 2, 4])
        B = rng.choice([1, 1, 2, 3])
        N = _log(rng, 1, min(524288, 500_000_000 // (B * (Hq + Hk) * d * es)))
        scaling = rng.choice(["none", "linear", "bands"])
        return {"op": op, "dtype": dtype, "B": B, "Hq": Hq, "Hk": Hk, "N": N, "d": d,
                "rot": rng.choice([d, d, d // 2, d // 4]), "layout": rng.choice(["half", "interleaved"]),
                "scaling": scaling, "base": rng.choice([10000.0, 500000.0]), "transpose": rng.random() < 0.5,
                "rows": rng.choice(["heads", "tokens"]), "packed": rng.random() < 0.4,
                "start": rng.choice([0, _log(rng, 1, 500000)])}
    page = rng.choice([16, 32, 64, 128])
    if op == "append":
        B = _log(rng, 1, 64)
        Hq = Hk * rng.choice([1, 2, 4])
        T = rng.choice([1, _log(rng, 2, max(2, min(32768, 300_000_000 // (B * (Hq + 2 * Hk) * d * es))))])
        most = max(T, min(65536, 600_000_000 // (B * Hk * d * es)))
        return {"op": op, "dtype": dtype, "B": B, "Hq": Hq, "Hk": Hk, "T": T, "d": d, "page": page,
                "length": _log(rng, T, most), "ragged": rng.random() < 0.5,
                "layout": rng.choice(["half", "interleaved"])}
    if op == "decode":
        B = _log(rng, 1, 128)
        Hq = Hk * rng.choice([1, 2, 3, 4, 8, 16])
        return {"op": op, "dtype": dtype, "B": B, "Hq": Hq, "Hk": Hk, "d": d, "page": page,
                "length": _log(rng, 1, min(524288, 500_000_000 // (B * Hk * d * es))),
                "ragged": rng.random() < 0.5, "weights": rng.random() < 0.3}
    B = _log(rng, 1, 32)
    n = _log(rng, 2, min(262144, 400_000_000 // (B * Hk * d * es)))
    budget = max(1, min(n, int(n * rng.uniform(0.2, 1.0))))
    return {"op": op, "dtype": dtype, "B": B, "Hk": Hk, "d": d, "page": page, "length": n, "budget": budget,
            "recent": rng.choice([0, budget // 8, budget // 2]), "ragged": rng.random() < 0.5,
            "positions": rng.random() < 0.5}


# --- what a program has in hand ---------------------------------------------------


def _lengths(case):
    """Sequence lengths: all equal, or spread from an empty one to the longest."""
    B, n = case["B"], case["length"]
    if not case["ragged"] or B == 1:
        return [n] * B
    return [n * ((7 * b) % B) // (B - 1) if math.gcd(7, B) == 1 else n * b // (B - 1) for b in range(B)]


def _counts(case):
    """New rows of each sequence of an append: all T, or fewer in a padded batch."""
    lens = _lengths(case)
    if not case["ragged"]:
        return [case["T"]] * case["B"]
    return [min(case["T"], n) for n in lens]


def _frequencies(case):
    rot = case.get("rot", case["d"])
    i = torch.arange(rot // 2, device=DEV, dtype=torch.float64)
    f = torch.exp(-math.log(case.get("base", 10000.0)) * (2.0 * i / rot))
    if case.get("scaling", "none") == "linear":
        f = f / 4.0
    elif case.get("scaling", "none") == "bands":
        turns = 8192.0 * f / (2.0 * math.pi)
        g = ((turns - 1.0) / (4.0 - 1.0)).clamp(0.0, 1.0)
        f = (1.0 - g) * f / 8.0 + g * f
    return f


def _plan(case):
    from long_context_hierarchical_b200 import lh
    more = {"none": {}, "linear": {"factor": 4.0},
            "bands": {"factor": 8.0, "low": 1.0, "high": 4.0, "original": 8192}}
    scaling = case.get("scaling", "none")
    return lh.rotary_plan(case["d"], rot=case.get("rot", case["d"]), base=case.get("base", 10000.0),
                          layout=case["layout"], scaling=scaling, **more[scaling])


def _normal(g, shape, dtype, scaled=True):
    """N(0, 1), times a lognormal scale for each row: the layer's own inputs."""
    x = torch.randn(shape, generator=g, device=DEV, dtype=torch.float32)
    if scaled:
        x.mul_(torch.exp(0.5 * torch.randn(shape[:-1] + (1,), generator=g, device=DEV)))
    return x.to(TYPES[dtype])


def _paged(case, g):
    """Pages in a random order, a table that points at them, and the sequences' lengths."""
    B, page = case["B"], case["page"]
    lens = _lengths(case)
    width = max(1, -(-max(lens) // page))
    used = [-(-n // page) for n in lens]
    total = max(1, sum(used))
    order = torch.randperm(total, generator=g, device=DEV, dtype=torch.int32)
    table = torch.zeros((B, width), device=DEV, dtype=torch.int32)
    col = torch.arange(width, device=DEV)
    mask = col[None, :] < torch.tensor(used, device=DEV)[:, None]
    table[mask] = order[: sum(used)]
    shape = (total, case["Hk"], page, case["d"])
    return {"k": _normal(g, shape, case["dtype"]), "v": _normal(g, shape, case["dtype"]), "table": table,
            "lengths": torch.tensor(lens, device=DEV, dtype=torch.int32)}


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    op, dtype, d = case["op"], case["dtype"], case["d"]
    s = {"case": case}
    if op == "rotary":
        B, N = case["B"], case["N"]
        for name, H in (("q", case["Hq"]), ("k", case["Hk"])):
            if case["rows"] == "tokens":
                s[name] = _normal(g, (B, N, H, d), dtype).transpose(1, 2)
            else:
                s[name] = _normal(g, (B, H, N, d), dtype)
        s["positions"] = None
        if case["packed"]:  # documents of odd lengths: positions begin again at each
            at = torch.arange(N, device=DEV, dtype=torch.int32)
            s["positions"] = torch.stack([case["start"] + (at + 57 * b) % (1021 + 2 * b) for b in range(B)]).int()
        s["f"] = _frequencies(case)
        if own:
            s["plan"] = _plan(case)
        return s
    s.update(_paged(case, g))
    if own:
        from long_context_hierarchical_b200 import lh
        s["cache"] = lh.PagedCache.of(s["k"], s["v"])
    if op == "append":
        B, T = case["B"], case["T"]
        s["new_q"] = _normal(g, (B, T, case["Hq"], d), dtype).transpose(1, 2)
        s["new_k"] = _normal(g, (B, T, case["Hk"], d), dtype).transpose(1, 2)
        s["new_v"] = _normal(g, (B, T, case["Hk"], d), dtype).transpose(1, 2)
        s["counts"] = torch.tensor(_counts(case), device=DEV, dtype=torch.int32) if case["ragged"] else None
        s["f"] = _frequencies(case)
        if own:
            s["plan"] = _plan(case)
    elif op == "decode":
        s["q"] = _normal(g, (case["B"], case["Hq"], 1, d), dtype)
        s["weights"] = None
        if case["weights"]:
            cap = s["table"].shape[1] * case["page"]
            at = torch.arange(cap, device=DEV)
            w = torch.exp(torch.randn((case["B"], case["Hk"], cap), generator=g, device=DEV) - 4.0)
            s["weights"] = torch.where(at < s["lengths"][:, None, None], w, 0.0)
            s["weights_out"] = torch.zeros_like(s["weights"])
    elif op == "evict":
        B, H = case["B"], case["Hk"]
        cap = s["table"].shape[1] * case["page"]
        at = torch.arange(cap, device=DEV, dtype=torch.int32)
        w = torch.exp(2.0 * torch.randn((B, H, cap), generator=g, device=DEV))
        # rows that no query has looked at yet weigh nothing: ties
        w = torch.where(torch.rand((B, H, cap), generator=g, device=DEV) < 0.02, 0.0, w)
        s["weights"] = torch.where(at < s["lengths"][:, None, None], w, 0.0)
        s["positions"] = None
        if case["positions"]:  # rows stand in the order that earlier evictions left
            key = torch.rand((B, H, cap), generator=g, device=DEV) + (at >= s["lengths"][:, None, None]) * 2.0
            s["positions"] = key.argsort(-1).argsort(-1).int()
        s["protect"] = (s["lengths"] - case["recent"]).int()
    return s


# --- one pass ----------------------------------------------------------------------


def run(state):
    op = state["case"]["op"]
    if own:
        return {"rotary": _own_rotary, "append": _own_append, "decode": _own_decode, "evict": _own_evict}[op](state)
    return {"rotary": _rotary, "append": _append, "decode": _decode, "evict": _evict}[op](state)


def _own_rotary(s):
    from long_context_hierarchical_b200 import lh
    call = lh.rotary_bwd if s["case"]["transpose"] else lh.rotary
    return call(s["plan"], s["q"], s["k"], positions=s["positions"], start=s["case"]["start"])


def _own_append(s):
    from long_context_hierarchical_b200 import lh
    q = lh.cache_append(s["cache"], s["table"], s["lengths"], s["new_k"], s["new_v"], Q=s["new_q"],
                        rotary=s["plan"], counts=s["counts"])
    return q, s["k"], s["v"]


def _own_decode(s):
    from long_context_hierarchical_b200 import lh
    if s["weights"] is None:
        return lh.decode(s["cache"], s["table"], s["lengths"], s["q"])
    o, lse = lh.decode(s["cache"], s["table"], s["lengths"], s["q"], weights=s["weights"],
                       weights_out=s["weights_out"])
    return o, lse, s["weights_out"]


def _own_evict(s):
    from long_context_hierarchical_b200 import lh
    n, w, p = lh.evict(s["cache"], s["table"], s["lengths"], s["weights"], s["case"]["budget"],
                       positions=s["positions"], protect=s["protect"])
    return (n, w, s["k"], s["v"]) if p is None else (n, w, s["k"], s["v"], p)


def _rotate(x, cos, sin, rot, layout):
    x = x.float()
    if layout == "half":
        a, b = x[..., : rot // 2], x[..., rot // 2: rot]
        y = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    else:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    return torch.cat((y, x[..., rot:]), -1)


def _rotary(s):
    c = s["case"]
    pos = s["positions"]
    if pos is None:
        pos = c["start"] + torch.arange(c["N"], device=DEV)[None]
    angle = pos[:, None, :, None].double() * s["f"]
    cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
    if c["transpose"]:
        sin = -sin
    return tuple(_rotate(s[x], cos, sin, c["rot"], c["layout"]).to(s[x].dtype) for x in ("q", "k"))


def _append(s):
    c = s["case"]
    T, page = c["T"], c["page"]
    n = s["lengths"].long()[:, None]
    count = (s["counts"].long() if s["counts"] is not None else torch.full_like(s["lengths"], T).long())[:, None]
    t = torch.arange(T, device=DEV)[None]
    slot = n - count + t
    there = t < count
    angle = slot[:, None, :, None].double() * s["f"]
    cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
    q = _rotate(s["new_q"], cos, sin, c["d"], c["layout"])
    q = torch.where(there[:, None, :, None], q, 0.0).to(s["new_q"].dtype)
    k = _rotate(s["new_k"], cos, sin, c["d"], c["layout"]).to(s["new_k"].dtype)
    b, at = there.nonzero(as_tuple=True)
    slot = slot[b, at]
    pages, row = s["table"].long()[b, slot // page], slot % page
    s["k"][pages, :, row] = k[b, :, at]
    s["v"][pages, :, row] = s["new_v"][b, :, at]
    return q, s["k"], s["v"]


def _rows(pages, table):
    """[B, H, width * page, d] of a paged tensor, in 32 bits."""
    x = pages[table.long()].float()
    B, w, H, page, d = x.shape
    return x.permute(0, 2, 1, 3, 4).reshape(B, H, w * page, d)


def _decode(s):
    c = s["case"]
    B, Hq, Hk, d = c["B"], c["Hq"], c["Hk"], c["d"]
    k, v = _rows(s["k"], s["table"]), _rows(s["v"], s["table"])
    there = (torch.arange(k.shape[2], device=DEV) < s["lengths"][:, None])[:, None, None]
    q = s["q"].float().reshape(B, Hk, Hq // Hk, d)
    x = (q @ k.transpose(2, 3)) * (1.0 / math.sqrt(d))
    x = torch.where(there, x, -math.inf)
    top = x.amax(-1, keepdim=True)
    safe = torch.where(top == -math.inf, 0.0, top)
    p = torch.exp(x - safe)
    total = p.sum(-1, keepdim=True)
    p = p / torch.where(total == 0, 1.0, total)
    o = (p @ torch.where(there.transpose(2, 3), v, 0.0)).reshape(B, Hq, 1, d).to(s["q"].dtype)
    lse = (safe + torch.log(total)).reshape(B, Hq, 1)
    if s["weights"] is None:
        return o, lse
    w = torch.where(there[:, :, 0], s["weights"] + p.sum(2), s["weights_out"])
    return o, lse, w


def _evict(s):
    c = s["case"]
    page, cap = c["page"], s["weights"].shape[-1]
    at = torch.arange(cap, device=DEV)
    n = s["lengths"].long()
    keep = torch.clamp(n, max=c["budget"])
    live = at < n[:, None, None]
    first = (at if s["positions"] is None else s["positions"]) >= s["protect"][:, None, None]
    rank = torch.where(live, torch.where(first, 2, 1), 0) * torch.ones_like(s["weights"], dtype=torch.int64)
    by_weight = torch.sort(s["weights"], dim=-1, descending=True, stable=True).indices
    by_rank = torch.sort(rank.gather(-1, by_weight), dim=-1, descending=True, stable=True).indices
    order = by_weight.gather(-1, by_rank)
    chosen = torch.zeros_like(rank).scatter(-1, order, (at < keep[:, None, None]).long().expand_as(order)) > 0
    low = at < keep[:, None, None]
    b, h, src = (chosen & ~low).nonzero(as_tuple=True)
    dst = (~chosen & low).nonzero(as_tuple=True)[2]
    table = s["table"].long()
    for x in ("k", "v"):
        s[x][table[b, dst // page], h, dst % page] = s[x][table[b, src // page], h, src % page]
    w = torch.where(low, s["weights"], 0.0)
    w[b, h, dst] = s["weights"][b, h, src]
    if s["positions"] is None:
        return keep.int(), w, s["k"], s["v"]
    p = torch.where(low, s["positions"], -1)
    p[b, h, dst] = s["positions"][b, h, src]
    return keep.int(), w, s["k"], s["v"], p


# --- what a pass cannot do without ----------------------------------------------------


def work(case):
    es, d, op = SIZE[case["dtype"]], case["d"], case["op"]
    if op == "rotary":
        rows = case["B"] * case["N"]
        heads = case["Hq"] + case["Hk"]
        return {"bytes": 2 * rows * heads * d * es + (4 * rows if case["packed"] else 0),
                "flops": 3 * rows * heads * case["rot"]}
    lens = _lengths(case)
    total = sum(lens)
    if op == "append":
        new = sum(_counts(case))
        padded = case["B"] * case["T"]
        return {"bytes": 2 * new * 2 * case["Hk"] * d * es + (new + padded) * case["Hq"] * d * es,
                "flops": 3 * new * (case["Hq"] + case["Hk"]) * d}
    if op == "decode":
        pages = sum(-(-n // case["page"]) for n in lens)
        return {"bytes": total * case["Hk"] * d * es * 2 + 2 * case["B"] * case["Hq"] * d * es + 4 * pages
                + (8 * total * case["Hk"] if case["weights"] else 0),
                "flops": 4 * total * case["Hq"] * d}
    width = -(-max(lens) // case["page"])
    moved = 0.0
    for n in lens:
        k = min(n, case["budget"])
        r = min(case["recent"], n, k)
        if n > k:
            spread = (k - r) * (n - k) / max(1, n - r)
            moved += spread + (0 if case["positions"] else r * (1.0 - (n - k) / max(1, n - r)))
    moved = int(moved) * case["Hk"]
    each = 4 * (2 if case["positions"] else 1)
    return {"bytes": each * case["Hk"] * (total + case["B"] * width * case["page"]) + 4 * moved * d * es,
            "flops": total * case["Hk"]}


# --- the definitions in 64 bits ---------------------------------------------------------


def _turn(x, pos, case, sign):
    """Pairs of channels as complex numbers, multiplied by exp(i angle)."""
    rot = case.get("rot", case["d"])
    x = x.double()
    pairs = x[..., :rot].unflatten(-1, (2, rot // 2)).transpose(-1, -2) if case["layout"] == "half" else \
        x[..., :rot].unflatten(-1, (rot // 2, 2))
    f = torch.tensor([_frequency(case, i) for i in range(rot // 2)], device=x.device, dtype=torch.float64)
    angle = sign * pos.double()[..., None] * f
    z = torch.view_as_complex(pairs.contiguous()) * torch.polar(torch.ones_like(angle), angle)
    pairs = torch.view_as_real(z)
    y = (pairs.transpose(-1, -2) if case["layout"] == "half" else pairs).flatten(-2)
    return torch.cat((y, x[..., rot:]), -1)


def _frequency(case, i):
    rot = case.get("rot", case["d"])
    f = case.get("base", 10000.0) ** (-2.0 * i / rot)
    kind = case.get("scaling", "none")
    if kind == "linear":
        return f / 4.0
    if kind == "bands":
        r = 8192.0 / (2.0 * math.pi / f)
        if r <= 1.0:
            return f / 8.0
        if r >= 4.0:
            return f
        g = (r - 1.0) / 3.0
        return (1.0 - g) * (f / 8.0) + g * f
    return f


def exact(case, seed):
    s = prepare(case, seed)
    op, d = case["op"], case["d"]
    if op == "rotary":
        pos = s["positions"] if s["positions"] is not None else \
            torch.arange(case["start"], case["start"] + case["N"], device=DEV).expand(case["B"], -1)
        sign = -1.0 if case["transpose"] else 1.0
        return tuple(_turn(s[x], pos[:, None], case, sign) for x in ("q", "k"))
    lens, page, table = _lengths(case), case["page"], s["table"].long()
    if op == "append":
        q = torch.zeros(s["new_q"].shape, device=DEV, dtype=torch.float64)
        k, v = s["k"].double(), s["v"].double()
        for b, m in enumerate(_counts(case)):
            if m:
                slot = torch.arange(lens[b] - m, lens[b], device=DEV)
                q[b, :, :m] = _turn(s["new_q"][b, :, :m], slot, case, 1.0)
                pages = table[b, torch.div(slot, page, rounding_mode="floor")]
                k[pages, :, slot % page] = _turn(s["new_k"][b, :, :m], slot, case, 1.0).transpose(0, 1)
                v[pages, :, slot % page] = s["new_v"][b, :, :m].double().transpose(0, 1)
        return q, k, v
    if op == "decode":
        B, Hq, Hk = case["B"], case["Hq"], case["Hk"]
        o = torch.zeros((B, Hq, 1, d), device=DEV, dtype=torch.float64)
        lse = torch.full((B, Hq, 1), -math.inf, device=DEV, dtype=torch.float64)
        w = s["weights_out"].double() if case["weights"] else None
        for b, n in enumerate(lens):
            if n == 0:
                continue
            own_pages = table[b, : -(-n // page)]
            k = s["k"][own_pages].transpose(0, 1).flatten(1, 2)[:, :n].double()
            v = s["v"][own_pages].transpose(0, 1).flatten(1, 2)[:, :n].double()
            q = s["q"][b].double().view(Hk, Hq // Hk, d)
            x = torch.einsum("hgd,hnd->hgn", q, k) / math.sqrt(d)
            total = torch.logsumexp(x, -1, keepdim=True)
            p = torch.exp(x - total)
            o[b] = torch.einsum("hgn,hnd->hgd", p, v).reshape(Hq, 1, d)
            lse[b] = total.reshape(Hq, 1)
            if w is not None:
                w[b, :, :n] = s["weights"][b, :, :n].double() + p.sum(1)
        return (o, lse) if w is None else (o, lse, w)
    # eviction computes no numbers: the weights that stay are moved, and follow from the definition
    w = s["weights"].double()
    out = torch.zeros_like(w)
    for b, n in enumerate(lens):
        m = min(n, case["budget"])
        for h in range(case["Hk"]):
            at = torch.arange(n, device=DEV)
            pos = at if s["positions"] is None else s["positions"][b, h, :n]
            prot = pos >= s["protect"][b]
            # one number that orders rows: protected before others, then the weight, then the lower slot
            level = torch.unique(w[b, h, :n], return_inverse=True)[1]
            key = (prot.long() * (n + 1) + level) * (n + 1) + (n - at)
            best = torch.argsort(key, descending=True)[:m].sort().values
            row = w[b, h, :m].clone()
            row_free = torch.ones(m, device=DEV, dtype=torch.bool)
            row_free[best[best < m]] = False
            row[row_free] = w[b, h, best[best >= m]]
            out[b, h, :m] = row
    none = [None, out, None, None]
    return tuple(none if s["positions"] is None else none + [None])
