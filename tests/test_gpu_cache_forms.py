"""Forms of the rotary and cache calls that their users meet, on the GPU: longer, wider and
repeated ones than the operators' own tests take.  Oracle and bounds are those of
tests/test_gpu_cache.py."""
import math
import os

import numpy as np
import pytest
import torch

from oracle import cache as oracle
from tests.helpers import np64
from tests.test_gpu_cache import U, Case, check_decode, gen, make_weights, normal

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("H,G", [(2, 1), (1, 8), (2, 12)])
@pytest.mark.parametrize("lens", [[37, 1, 0, 200], [1500, 64]])
def test_decode_rounds_only_what_it_stores(d, H, G, lens):
    """bf16 outputs are as good as fp32 probabilities make them.  A probability enters
    the product as two bf16 numbers: the first is within 2^-8 of it, the remainder is
    exact in fp32 and the second within 2^-8 of that, so together they are within 2^-16
    of the probability.  |O - o| <= T (2 ds + 2^-16 + (2 n_chain + 32 + S) u) + H |o| in
    the header's terms, for every channel, small ones among them."""
    from long_context_hierarchical_b200 import lh
    c = Case(lens, H, d, 16, "bf16", seed=d + G)
    q = normal(c.g, (len(lens), H * G, 1, d), "bf16")
    o, _ = lh.decode(c.cache, c.table, c.lengths, q)
    for b, n in enumerate(lens):
        if n == 0:
            continue
        k, v, qb = np64(c.rows(c.k, b)), np64(c.rows(c.v, b)), np64(q[b, :, 0])
        want, lse, p = oracle.decode(qb, k, v, d ** -0.5)
        kr, vr = np.repeat(k, G, 0), np.repeat(v, G, 0)
        ds = (d + 6) * U * d ** -0.5 * np.einsum("hd,hnd->hn", np.abs(qb), np.abs(kr)).max(1)
        S = np.abs(np.einsum("hd,hnd->hn", qb, kr) * d ** -0.5 - lse[:, None]).max(1) / math.log(2.0) + 8
        rel = 2 * ds + 2.0 ** -16 + (2 * (n / 8 + 664) + 32 + S) * U
        tol = np.einsum("hn,hnd->hd", p, np.abs(vr)) * rel[:, None] + 2.0 ** -8 * np.abs(want) * (1 + 2.0 ** -7)
        off = np.abs(np64(o[b, :, 0]) - want)
        assert np.all(off <= tol), (b, (off / tol).max())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d,G", [(64, 1), (128, 3), (64, 16)])
def test_decode_carries_an_infinite_value(dtype, d, G):
    """An infinity among the values attended to is the output of its channel, with its sign
    (a positive probability times it), infinities of both signs a NaN; other channels are as without it."""
    from long_context_hierarchical_b200 import lh
    c = Case([200, 5], 2, d, 16, dtype, seed=G)
    q = normal(c.g, (2, 2 * G, 1, d), dtype)
    want = lh.decode(c.cache, c.table, c.lengths, q)
    for b, j, h, ch, x in ((0, 3, 0, 1, math.inf), (0, 150, 0, 2, -math.inf), (0, 199, 0, 2, -math.inf),
                           (0, 60, 0, 40, math.inf), (0, 61, 0, 40, -math.inf), (1, 0, 1, 5, -math.inf)):
        c.v[int(c.table[b, j // 16]), h, j % 16, ch] = x
    o, lse = lh.decode(c.cache, c.table, c.lengths, q)
    assert torch.equal(lse, want[1])
    assert bool((o[0, :G, 0, 1] == math.inf).all()) and bool((o[0, :G, 0, 2] == -math.inf).all())
    assert torch.isnan(o[0, :G, 0, 40]).all() and bool((o[1, G:, 0, 5] == -math.inf).all())
    for b, heads, channels in ((0, slice(0, G), [1, 2, 40]), (1, slice(G, 2 * G), [5])):
        o[b, heads, 0, channels] = want[0][b, heads, 0, channels]
    assert torch.equal(o, want[0])


def test_layer_with_rotary_keeps_the_shape_of_its_queries():
    """O has the shape of Q, with rotary as without it."""
    from long_context_hierarchical_b200 import lh
    g = gen(7)
    B, H, N, d = 2, 3, 128, 64
    pl = lh.plan(B, H, N, d, 4, 3, 4, "bf16")
    rp = lh.rotary_plan(d)
    Q, K, V = (normal(g, (B, H, N, d), "bf16") for _ in range(3))
    want = lh.forward(pl, Q, K, V, rotary=rp)[0]
    for shape in ((B * H, N, d), (B * H * N, d), (-1,)):
        for k in (K, K.view(B * H, N, d)):
            assert lh.forward(pl, Q.view(shape), k, V)[0].shape == Q.view(shape).shape
            O = lh.forward(pl, Q.view(shape), k, V, rotary=rp)[0]
            assert O.shape == Q.view(shape).shape and torch.equal(O.view(B, H, N, d), want)


def test_readme_answering_example_over_many_steps():
    """The README's steps (append, decode, evict), repeated as they stand with small sizes: what
    is left in the cache are rows of the sequence turned at their own positions, the
    newest among them, and the answer is dense attention over exactly these rows."""
    from long_context_hierarchical_b200 import lh
    text = open(os.path.join(os.path.dirname(os.path.dirname(__file__)), "README.md")).read()
    block = next(x for x in text.split("```python\n")[1:] if "lh.cache_append" in x).split("```")[0]
    B, H, d, page, width, budget, recent = 2, 2, 64, 16, 4, 40, 8
    for a, b in (("49152", str(budget)), ("1024", str(recent)), ("4096", str(B * width)), ("page=64", f"page={page}"),
                 ("H=16", f"H={H}")):
        assert a in block
        block = block.replace(a, b)
    first, steps = block.split("\n", 1)
    assert "PagedCache" in first
    g = gen(14)
    cap = width * page
    i32 = dict(dtype=torch.int32, device="cuda")
    env = dict(lh=lh, torch=torch, rp=lh.rotary_plan(d, base=500000.0), B=B,
               table=torch.randperm(B * width, generator=g, **i32).view(B, width), lengths=torch.zeros(B, **i32),
               seen=torch.zeros(B, **i32), weights=torch.zeros((B, H, cap), device="cuda"),
               slot_positions=torch.full((B, H, cap), -1, **i32))
    exec(first, env)
    cache, total = env["cache"], 0
    keys = torch.empty((B, H, 0, d), dtype=torch.bfloat16, device="cuda")   # of all rows so far, turned
    values = keys.clone()
    for T in [30, 1, 25, 1, 1, 20] + [1] * 20:
        env["T"] = T
        env["K"], env["V"], env["Q"] = (normal(g, (B, H, T, d), "bf16") for _ in range(3))
        q = lh.rotary(env["rp"], env["Q"], start=total)[:, :, -1:]
        keys = torch.cat((keys, lh.rotary(env["rp"], env["K"], start=total)), 2)
        values = torch.cat((values, env["V"]), 2)
        total += T
        exec(steps, env)
        for b in range(B):
            n = int(env["lengths"][b])
            assert n == min(total, budget)
            at = torch.arange(n, device="cuda")
            ids = env["table"][b].long()[at // page]
            for h in range(H):
                k, v = cache.k[ids, h, at % page], cache.v[ids, h, at % page]
                same = (v[:, None] == values[b, h][None]).all(-1)       # which row stands in which slot
                assert bool((same.sum(1) == 1).all())
                row = same.int().argmax(1)
                assert torch.equal(k, keys[b, h, row])                 # turned at its own position
                kept = set(row.tolist())
                assert len(kept) == n and set(range(total - min(recent, n), total)) <= kept
        if total == T:   # the first step: every row was there
            for b in range(B):
                wo, _, p = oracle.decode(np64(q[b, :, 0]), np64(keys[b]), np64(values[b]), d ** -0.5)
                T_o = np.einsum("hn,hnd->hd", p, np.abs(np64(values[b])))
                assert np.all(np.abs(np64(env["O"][b, :, 0]) - wo) <= 2.0 ** -6 * (T_o + np.abs(wo)))
    lh.device_status()


def check_evicted_heads(c, heads, budget, w0, p0, protect, got, k0, v0):
    """Some heads of a single sequence: weights, positions and rows."""
    table = c.table[0].long()
    for h in heads:
        _, moves, _ = oracle.evict(w0[0, h].cpu().numpy(), c.lens[0], budget,
                                   None if p0 is None else p0[0, h].cpu().numpy(), protect)
        src, dst = (torch.tensor(x, device="cuda") for x in zip(*moves))
        want = torch.zeros(c.capacity, device="cuda")
        want[:budget] = w0[0, h, :budget]
        want[dst] = w0[0, h, src]
        assert torch.equal(got[1][0, h], want)
        if p0 is not None:
            p = torch.full((c.capacity,), -1, dtype=torch.int32, device="cuda")
            p[:budget] = p0[0, h, :budget]
            p[dst] = p0[0, h, src]
            assert torch.equal(got[2][0, h], p)
        for x, x0 in ((c.k, k0), (c.v, v0)):
            rows = x0[:, h].clone()
            rows[table[dst // c.page], dst % c.page] = x0[table[src // c.page], h, src % c.page]
            assert torch.equal(x[:, h].nan_to_num(9.0), rows.nan_to_num(9.0))


@pytest.mark.parametrize("H,n,budget,protected,placed,in_place", [
    *[(1, 330003, 100000, a, b, c) for a in (False, True) for b in (False, True) for c in (False, True)],
    *[(H, n, n // 2, a, a, c) for H, n in ((80, 41003), (50, 82003)) for a in (False, True) for c in (False, True)]])
def test_evict_reads_weights_again_where_keys_do_not_fit(H, n, budget, protected, placed, in_place):
    """A block keeps the keys of at most 40960 slots in shared memory and at most eight
    blocks share a head, so 330,003 slots never fit, however many blocks a head gets; where 148 SMs
    are one block a head (two), 41,003 (82,003) slots do not either."""
    from long_context_hierarchical_b200 import lh
    assert n > 40960 * min(8, 148 // H)
    c = Case([n], H, 64, 256, "bf16", seed=6)
    w = make_weights(c, "ties" if protected else "spread")
    w[:, :, n:] = 0.0
    pos = torch.rand(w.shape, generator=c.g, device="cuda").argsort(-1).int() if placed else None
    first = n - n // 4
    protect = torch.tensor([first], dtype=torch.int32, device="cuda") if protected else None
    k0, v0 = c.k.clone(), c.v.clone()
    w0, p0 = w.clone(), None if pos is None else pos.clone()
    got = lh.evict(c.cache, c.table, c.lengths, w, budget, positions=pos, protect=protect,
                   weights_out=w if in_place else None, positions_out=pos if in_place else None)
    assert int(got[0][0]) == budget
    check_evicted_heads(c, (0,) if H == 1 else (0, H - 1), budget, w0, p0, first if protected else None, got, k0, v0)
    lh.device_status()


@pytest.mark.parametrize("dtype,d,Hq,H,T", [("bf16", 64, 9, 3, 20001), ("bf16", 64, 6, 3, 40001),
                                            ("bf16", 128, 2, 1, 20001), ("bf16", 128, 9, 3, 10001),
                                            ("f32", 64, 2, 1, 40001), ("f32", 128, 4, 2, 20001)])
def test_append_blocks_of_several_heads(dtype, d, Hq, H, T):
    """Rows enough that a block takes several heads (all of them, or a part that begins
    and ends inside Q, K or V): a pair of heads in flight is the last of Q and the first of K, or
    the last of K and the first of V, and the last is alone.  The bits are those of lh.rotary and of
    copies; padding is not read and nothing else is written."""
    from long_context_hierarchical_b200 import lh
    counts = [T, T // 2 + 3, T - 1]
    lens = [counts[0] + 5, counts[1], counts[2] + 100]
    c = Case(lens, H, d, 64, dtype, seed=Hq, width=-(-max(lens) // 64) + 1)
    k0, v0 = c.k.nan_to_num(9.0), c.v.nan_to_num(9.0)
    q = normal(c.g, (3, T, Hq, d), dtype).transpose(1, 2)
    k, v = (normal(c.g, (3, H, T, d), dtype) for _ in range(2))
    for b, m in enumerate(counts):   # padding that would show
        for x in (q, k, v):
            x[b, :, m:] = float("nan")
    cnt = torch.tensor(counts, dtype=torch.int32, device="cuda")
    given = torch.randint(0, 500000, (3, T), generator=c.g, device="cuda", dtype=torch.int32)
    slots = ((c.lengths - cnt)[:, None] + torch.arange(T, device="cuda", dtype=torch.int32)).int()
    for rp, positions in ((lh.rotary_plan(d, rot=d // 2), None), (lh.rotary_plan(d, layout="interleaved"), given),
                          (None, None)):
        c.k.copy_(k0)
        c.v.copy_(v0)
        sp = torch.full((3, H, c.capacity), -9, dtype=torch.int32, device="cuda")
        pos = slots if positions is None else positions
        want_q, want_k = (q, k) if rp is None else lh.rotary(rp, q, k, positions=pos)
        qi = q.clone()
        out = lh.cache_append(c.cache, c.table, c.lengths, k, v, Q=qi, rotary=rp, positions=positions, counts=cnt,
                              slot_positions=sp, out=qi)
        assert out is qi
        again = lh.cache_append(c.cache, c.table, c.lengths, k, v, Q=q, rotary=rp, positions=positions, counts=cnt)
        assert torch.equal(again, qi)
        k1, v1, sp1 = k0.clone(), v0.clone(), torch.full_like(sp, -9)
        for b, m in enumerate(counts):
            assert torch.equal(qi[b, :, :m], want_q[b, :, :m]) and not qi[b, :, m:].any()
            at = slots[b, :m].long()
            page, row = c.table[b].long()[at // 64], at % 64
            k1[page, :, row] = want_k[b, :, :m].transpose(0, 1)
            v1[page, :, row] = v[b, :, :m].transpose(0, 1)
            sp1[b, :, at] = pos[b, :m]
        assert torch.equal(c.k, k1) and torch.equal(c.v, v1) and torch.equal(sp, sp1)
    lh.device_status()


@pytest.mark.parametrize("dtype,d,Hq", [("bf16", 64, 3), ("f32", 64, 1), ("bf16", 128, 2), ("f32", 128, 1)])
@pytest.mark.parametrize("n", [4096, 4097, 8192, 8193, 300001])
def test_decode_join_of_many_parts(dtype, d, Hq, n):
    """One key head, no weights: as many parts as tiles of 64 slots (64, 65, 128, 129) or
    blocks (hundreds) are joined by the launch for few heads.  Its bits are those of the
    launch that joins beside the weights."""
    from long_context_hierarchical_b200 import lh
    c = Case([n], 1, d, 1024, dtype, seed=n % 97)
    q = normal(c.g, (1, Hq, 1, d), dtype)
    o, lse = lh.decode(c.cache, c.table, c.lengths, q)
    check_decode(c, q, o, lse)
    w = torch.zeros((1, 1, c.capacity), device="cuda")
    o2, lse2 = lh.decode(c.cache, c.table, c.lengths, q, weights=w)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    check_decode(c, q, o, lse, weights=torch.zeros_like(w), weights_out=w)
