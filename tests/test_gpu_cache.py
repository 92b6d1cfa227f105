"""Rotary positions, cache append, decoding attention and eviction on the GPU,
against the fp64 oracle (oracle/cache.py).

Bounds, all derived from the arithmetic (u = 2^-24, one fp32 rounding; H =
eps/2 of the storage type, one rounding to it):

  rotary   The angle in half turns is rounded once (u of at most 1, so pi u in
           radians), sincospi is within 2 u of a value of at most 1, the
           magnitude one more: a sine or cosine is within 7 u m.  Two products
           and a sum round by at most 2 u (|a| + |b|) m.  Total 9 u m (|a| +
           |b|), plus the oracle's own angle, off by 2^-52 |t f|, plus H |y|
           for the storage type.
  decode   A score is d products of fp32 (bf16 products are exact) in a chain
           of at most d sums, q scaled once before or the score after: within
           (d + 6) u A of itself, A = scale max_j sum_c |q_c k_jc|; call it ds
           (nats).  exp2 of a difference of such numbers: relative 2 ds +
           8 u + u max|s - lse| ; a probability is rounded to the storage type
           where it is a bf16 MMA operand (H).  l and O are sums of positive
           weights times values, in a chain of at most n + 64 sums.  So
           |O - o| <= T (2 ds + H + (2 n_chain + 32) u + S u) + H |o|,
           T = sum p |v|, S = max |s - lse| * log2(e) + 8, and lse within
           ds + (n_chain + 16) u + 4 u |lse|.  n_chain: one lane sums at most
           n / 8 keys, and the parts of all ranges.
           That worst case would hide a single key left out of a long sequence, so
           each row is also held in L2 norm: the roundings of the probabilities are
           independent and spread by 2^-8 / sqrt(3) of themselves, those of the output
           are at most H, so |O - o| <= 4 |sigma| + H |o| + |T| (the fp32 terms above)
           with sigma_c = 2^-8 / sqrt(3) (sum_j (p_j v_jc)^2)^(1/2).
  weights  Sum of G probabilities: (2 ds + d_lse + (S + 16) u) sum p + 2 u |w + sum p|.
  evict    No arithmetic: equal.
"""
import math

import numpy as np
import pytest
import torch

from oracle import cache as oracle
from tests.helpers import np64

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def normal(g, shape, dtype):
    x = torch.randn(shape, generator=g, device="cuda")
    return (x * torch.exp(0.5 * torch.randn(shape[:-1] + (1,), generator=g, device="cuda"))).to(DT[dtype])


# --- rotary -----------------------------------------------------------------------


def check_rotary(got, x, pos, f, layout, m=1.0, transpose=False, pos_axes=True):
    """got, x: [B, H, N, d] tensors; pos: [B, N] or [1, N] numpy."""
    xs = np64(x)
    p = pos[:, None, :]
    want = oracle.rotate(xs, p, f, layout, m, transpose)
    rot = 2 * len(f)
    mate = np.abs(xs)
    if layout == "half":
        mate[..., : rot // 2] += np.abs(xs[..., rot // 2: rot])
        mate[..., rot // 2: rot] = mate[..., : rot // 2]
    else:
        pair = np.abs(xs[..., 0:rot:2]) + np.abs(xs[..., 1:rot:2])
        mate[..., 0:rot:2] = mate[..., 1:rot:2] = pair
    far = 2.0 ** -52 * np.abs(pos).max() * f.max()
    tol = (9 * U + far) * m * mate + HALF[x.dtype] * np.abs(want) * (1 + 2.0 ** -7)
    g = np64(got)
    assert got.dtype == x.dtype and got.shape == x.shape
    assert np.isfinite(g).all()
    off = np.abs(g - want)
    assert np.all(off <= tol), (off - tol).max()
    assert np.array_equal(g[..., rot:], xs[..., rot:])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d,rot,layout", [(64, 64, "half"), (64, 16, "half"), (64, 32, "interleaved"),
                                          (128, 128, "interleaved"), (128, 96, "half"), (128, 16, "interleaved")])
@pytest.mark.parametrize("B,Hq,Hk,N", [(1, 1, 1, 1), (2, 3, 1, 67), (3, 5, 2, 1)])
def test_rotary_shapes(dtype, d, rot, layout, B, Hq, Hk, N):
    from long_context_hierarchical_b200 import lh
    g = gen(B * 100 + N)
    q, k = normal(g, (B, Hq, N, d), dtype), normal(g, (B, Hk, N, d), dtype)
    rp = lh.rotary_plan(d, rot=rot, layout=layout)
    f = oracle.frequencies(rot)
    pos = np.arange(N)[None] + 11
    for call, t in ((lh.rotary, False), (lh.rotary_bwd, True)):
        a, b = call(rp, q, k, start=11)
        check_rotary(a, q, pos, f, layout, transpose=t)
        check_rotary(b, k, pos, f, layout, transpose=t)
        assert torch.equal(call(rp, q, start=11), a)   # alone: the same bits


@pytest.mark.parametrize("dtype,d,Hq,Hk,N", [("bf16", 64, 7, 3, 120001), ("bf16", 64, 17, 1, 120001),
                                             ("bf16", 128, 9, 2, 60001), ("f32", 64, 5, 2, 120001),
                                             ("f32", 128, 3, 8, 60001)])
def test_rotary_blocks_of_several_heads(dtype, d, Hq, Hk, N):
    # rows enough for blocks of several heads, some of Q's last and K's first: the bits
    # of each head turned alone, also in place
    from long_context_hierarchical_b200 import lh
    g = gen(Hq)
    rp = lh.rotary_plan(d, rot=d // 2)
    q, k = normal(g, (1, Hq, N, d), dtype), normal(g, (1, Hk, N, d), dtype)
    turned = lh.rotary(rp, q, k, start=7)
    for x, y in zip((q, k), turned):
        for h in range(x.shape[1]):
            assert torch.equal(y[:, h:h + 1], lh.rotary(rp, x[:, h:h + 1], start=7)), h
    lh.rotary(rp, q, k, start=7, out=(q, k))
    assert torch.equal(q, turned[0]) and torch.equal(k, turned[1])


@pytest.mark.parametrize("kw", [
    dict(scaling="linear", factor=4.0), dict(scaling="bands", factor=8.0, low=1.0, high=4.0, original=8192.0),
    dict(magnitude=1.25), dict(base=500000.0)])
def test_rotary_scalings_and_far_positions(kw):
    from long_context_hierarchical_b200 import lh
    g = gen(3)
    x = normal(g, (2, 2, 9, 64), "f32")
    pos = torch.tensor([[0, 1, 524287, 2 ** 31 - 1, -1, -2 ** 31, 98303, 7, 7],
                        [1 << 24, (1 << 24) + 1, 3, 2, 1, 0, -5, 1 << 30, 65537]], dtype=torch.int32, device="cuda")
    rp = lh.rotary_plan(64, **kw)
    m = kw.pop("magnitude", 1.0)
    f = oracle.frequencies(64, **kw)
    got = lh.rotary(rp, x, positions=pos)
    check_rotary(got, x, np64(pos), f, "half", m)
    # a shared row of positions, as [N] and as [1, N]
    for p in (pos[1].contiguous(), pos[1:]):
        check_rotary(lh.rotary(rp, x, positions=p), x, np64(pos[1:]), f, "half", m)


def test_rotary_strides_and_places():
    from long_context_hierarchical_b200 import lh
    g = gen(4)
    rp = lh.rotary_plan(64)
    f = oracle.frequencies(64)
    B, H, N = 2, 4, 33
    pos = np.arange(N)[None]
    # a fused projection [B, N, 3, H, d]: q and k slices, in place
    fused = normal(g, (B, N, 3, H, 64), "bf16")
    before = fused.clone()
    q, k = fused[:, :, 0].transpose(1, 2), fused[:, :, 1].transpose(1, 2)
    want = lh.rotary(rp, q, k)
    assert want[0].is_contiguous()
    check_rotary(want[0], q, pos, f, "half")
    got = lh.rotary(rp, q, k, out=(q, k))
    assert got[0] is q
    assert torch.equal(q, want[0]) and torch.equal(k, want[1])
    assert torch.equal(fused[:, :, 2], before[:, :, 2])
    # a broadcast input: one head's rows for all heads
    one = normal(g, (B, 1, N, 64), "bf16")
    assert torch.equal(lh.rotary(rp, one.expand(B, H, N, 64)), lh.rotary(rp, one).expand(B, H, N, 64))
    # rows behind the ones of the call stay as they are
    room = torch.full((B, H, N + 5, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    x = normal(g, (B, H, N, 64), "bf16")
    lh.rotary(rp, x, out=room[:, :, :N])
    assert torch.equal(room[:, :, :N], lh.rotary(rp, x)) and bool((room[:, :, N:] == 7.0).all())
    assert lh.rotary(rp, x[:, :, :0]).shape == (B, H, 0, 64)
    with pytest.raises(lh.LighthouseError):
        lh.rotary(rp, x[:, :, :-1], out=x[:, :, 1:])   # shifted by a row
    with pytest.raises(lh.LighthouseError):
        lh.rotary(rp, x, out=one.expand(B, H, N, 64))  # rows on one another


def test_rotary_rows_off_the_boundary_are_refused():
    from long_context_hierarchical_b200 import lh
    flat = torch.zeros(2 * 3 * 65, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(lh.LighthouseError) as e:
        lh.rotary(lh.rotary_plan(64), flat.view(1, 2, 3, 65)[..., :64])
    assert e.value.status == lh.LH_ERR_INVALID_ARG


def test_rotary_gradient_against_differences():
    """L = <g, rotary(x)> is linear in x, so a central difference of any step is
    exact up to rounding: |dL/dx_i - (L(x + h) - L(x - h)) / 2h| with h = 1, the
    sums in fp64 over fp32 outputs, each off by 9 u (|a| + |b|)."""
    from long_context_hierarchical_b200 import lh
    g = gen(5)
    x, go = normal(g, (1, 2, 5, 64), "f32"), normal(g, (1, 2, 5, 64), "f32")
    for layout in ("half", "interleaved"):
        rp = lh.rotary_plan(64, rot=32, layout=layout, magnitude=1.1)
        grad = lh.rotary_bwd(rp, go, start=1000)
        for n, h, c in ((0, 0, 0), (4, 1, 31), (2, 0, 16), (3, 1, 40)):
            up, down = x.clone(), x.clone()
            up[0, h, n, c] += 1.0
            down[0, h, n, c] -= 1.0
            loss = [(lh.rotary(rp, y, start=1000).double() * go.double()).sum().item() for y in (up, down)]
            size = 4 * 9 * U * 1.1 * (x.abs()[0, h, n].max().item() + 1) * go.abs()[0, h, n].max().item()
            assert abs(grad[0, h, n, c].item() - (loss[0] - loss[1]) / 2) <= size + 9 * U * 2.2 * go.abs().max().item()


@pytest.mark.parametrize("dtype,d", [("bf16", 64), ("f32", 64), ("bf16", 128)])
def test_layer_with_rotary_is_the_layer_on_turned_inputs(dtype, d):
    from long_context_hierarchical_b200 import lh
    g = gen(6)
    B, H, N = 2, 2, 256
    pl = lh.plan(B, H, N, d, 4, 3, 4, dtype)
    Q, K, V, dO = (normal(g, (B, H, N, d), dtype) for _ in range(4))
    keep = Q.clone(), K.clone()
    rp = lh.rotary_plan(d)
    pos = (torch.arange(N, device="cuda", dtype=torch.int32) % 100).repeat(B, 1)
    for kw in (dict(start=77), dict(positions=pos)):
        lh.set_deterministic(True)
        try:
            O, ctx = lh.forward(pl, Q, K, V, rotary=rp, **kw)
            got = lh.backward(pl, dO, ctx)
            Qr, Kr = lh.rotary(rp, Q, K, **kw)
            O2, ctx2 = lh.forward(pl, Qr, Kr, V)
            dQ, dK, dV = lh.backward(pl, dO, ctx2)
        finally:
            lh.set_deterministic(False)
        assert torch.equal(O, O2) and torch.equal(got[2], dV)
        dQ, dK = lh.rotary_bwd(rp, dQ, dK, **kw)
        assert torch.equal(got[0], dQ) and torch.equal(got[1], dK)
        assert torch.equal(Q, keep[0]) and torch.equal(K, keep[1])
    # a context that is used again without rotary no longer turns
    O3, ctx = lh.forward(pl, Q, K, V, ctx=ctx)
    assert ctx.rotary is None


# --- cache ---------------------------------------------------------------------------


class Case:
    """A cache of `lens` rows on shuffled pages; pages that nothing points at hold NaN."""

    def __init__(self, lens, H, d, page, dtype, seed=0, width=None, spare=2):
        g = gen(seed)
        used = [-(-n // page) for n in lens]
        width = width or max(1, max(used))
        total = sum(used) + spare
        order = torch.randperm(total, generator=g, device="cuda", dtype=torch.int32)
        self.table = torch.full((len(lens), width), int(order[-1]), dtype=torch.int32, device="cuda")
        self.k = torch.full((total, H, page, d), float("nan"), device="cuda", dtype=DT[dtype])
        self.v = self.k.clone()
        at = 0
        for b, n in enumerate(lens):
            ids = order[at: at + used[b]]
            at += used[b]
            self.table[b, : used[b]] = ids
            for x in (self.k, self.v):
                row = normal(g, (H, used[b] * page, d), dtype)
                row[:, n:] = float("nan")   # behind the length
                x[ids.long()] = row.view(H, used[b], page, d).transpose(0, 1)
        self.lens, self.H, self.d, self.page, self.width = list(lens), H, d, page, width
        self.capacity = width * page
        self.lengths = torch.tensor(list(lens), dtype=torch.int32, device="cuda")
        from long_context_hierarchical_b200 import lh
        self.cache = lh.PagedCache.of(self.k, self.v)
        self.g = g
        self.dtype = dtype

    def rows(self, x, b, n=None):
        n = self.lens[b] if n is None else n
        ids = self.table[b].long()[: -(-n // self.page)]
        return x[ids].transpose(0, 1).reshape(self.H, -1, self.d)[:, :n]


def check_decode(c, q, o, lse, scale=None, weights=None, weights_out=None, bad=()):
    d, dt = c.d, DT[c.dtype]
    scale = d ** -0.5 if scale is None else scale
    Hq = q.shape[1]
    G = Hq // c.H
    for b, n in enumerate(c.lens):
        k, v = np64(c.rows(c.k, b)), np64(c.rows(c.v, b))
        live = np.array([j for j in range(n) if (b, j // c.page) not in bad], dtype=int)
        k, v = k[:, live], v[:, live]
        qb = np64(q[b, :, 0])
        wo, wl, p = oracle.decode(qb, k, v, scale)
        go, gl = np64(o[b, :, 0]), np64(lse[b, :, 0])
        if len(live) == 0:
            assert not go.any() and np.isneginf(gl).all()
            continue
        kr, vr = np.repeat(k, G, 0), np.repeat(v, G, 0)
        A = abs(scale) * np.einsum("hd,hnd->hn", np.abs(qb), np.abs(kr)).max(1)
        s = np.einsum("hd,hnd->hn", qb, kr) * scale
        S = (np.abs(s - wl[:, None]).max(1)) / math.log(2.0) + 8
        ds = (d + 6) * U * A
        chain = n / 8 + 64 + 600
        T = np.einsum("hn,hnd->hd", p, np.abs(vr))
        rel = 2 * ds + (HALF[dt] if dt == torch.bfloat16 else 0.0) + (2 * chain + 32) * U + S * U
        tol = T * rel[:, None] + HALF[dt] * np.abs(wo) * (1 + 2.0 ** -7)
        assert np.isfinite(go).all()
        assert np.all(np.abs(go - wo) <= tol), (b, np.abs(go - wo).max())
        spread = 2.0 ** -8 / math.sqrt(3.0) if dt == torch.bfloat16 else 0.0
        sigma = spread * np.sqrt(np.einsum("hn,hnd->hd", p * p, vr * vr))
        norm = lambda x: np.linalg.norm(x, axis=1)  # noqa: E731
        fp32 = 2 * ds + (2 * chain + 32) * U + S * U
        row = 4 * norm(sigma) + HALF[dt] * norm(wo) * (1 + 2.0 ** -7) + norm(T) * fp32
        assert np.all(norm(go - wo) <= row), (b, (norm(go - wo) / row).max())
        dl = ds + (chain + 16) * U + 4 * U * np.abs(wl)
        assert np.all(np.abs(gl - wl) <= dl), (b, np.abs(gl - wl).max())
        if weights is not None:
            ps = p.reshape(c.H, G, -1).sum(1)
            w0, w1 = np64(weights[b]), np64(weights_out[b])
            prel = (2 * ds + dl + (S + 16) * U).reshape(c.H, G).max(1)
            want = w0[:, live] + ps
            assert np.all(np.abs(w1[:, live] - want) <= prel[:, None] * ps + 2 * U * np.abs(want)), b


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("H,G", [(1, 1), (2, 2), (2, 3), (1, 7), (2, 8), (1, 12), (1, 16), (2, 17), (1, 40)])
def test_decode_heads(dtype, d, H, G):
    from long_context_hierarchical_b200 import lh
    c = Case([70, 1, 0, 257], H, d, 16, dtype, seed=G)
    q = normal(c.g, (4, H * G, 1, d), dtype)
    o, lse = lh.decode(c.cache, c.table, c.lengths, q)
    assert o.shape == (4, H * G, 1, d) and lse.shape == (4, H * G, 1) and o.dtype == DT[dtype]
    check_decode(c, q, o, lse)
    w = torch.rand((4, H, c.capacity), generator=c.g, device="cuda")
    out = torch.full_like(w, -5.0)
    o2, lse2 = lh.decode(c.cache, c.table, c.lengths, q, weights=w, weights_out=out)
    assert torch.equal(o2, o) and torch.equal(lse2, lse)
    check_decode(c, q, o, lse, weights=w, weights_out=out)
    for b, n in enumerate(c.lens):
        assert bool((out[b, :, n:] == -5.0).all())       # behind the length: untouched
    w2 = w.clone()
    lh.decode(c.cache, c.table, c.lengths, q, weights=w2)  # in place
    for b, n in enumerate(c.lens):
        assert torch.equal(w2[b, :, :n], out[b, :, :n]) and torch.equal(w2[b, :, n:], w[b, :, n:])
    lh.device_status()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("page", [16, 64, 256])
@pytest.mark.parametrize("lens", [[1], [15, 16, 17], [63, 64, 65, 0, 0, 127], [5000], [0, 0], [4096, 3, 900, 0, 33]])
def test_decode_lengths_and_pages(dtype, page, lens):
    from long_context_hierarchical_b200 import lh
    c = Case(lens, 2, 64, page, dtype, seed=len(lens), width=-(-max(lens + [1]) // page) + 3)
    q = normal(c.g, (len(lens), 4, 1, 64), dtype)
    w = torch.zeros((len(lens), 2, c.capacity), device="cuda")
    out = torch.zeros_like(w)
    o, lse = lh.decode(c.cache, c.table, c.lengths, q, weights=w, weights_out=out)
    check_decode(c, q, o, lse, weights=w, weights_out=out)
    lh.device_status()


@pytest.mark.parametrize("dtype,d,Hq", [("bf16", 64, 3), ("f32", 64, 1), ("bf16", 128, 12), ("f32", 128, 2)])
def test_decode_long(dtype, d, Hq):
    from long_context_hierarchical_b200 import lh
    c = Case([300001, 1], 1, d, 1024, dtype, seed=d)
    q = normal(c.g, (2, Hq, 1, d), dtype)
    w = torch.zeros((2, 1, c.capacity), device="cuda")
    o, lse = lh.decode(c.cache, c.table, c.lengths, q, weights=w)
    check_decode(c, q, o, lse, weights=torch.zeros_like(w), weights_out=w)


def test_decode_many_sequences_and_order_free():
    """More sequences than a warp holds lengths, most ranges over several of
    them; a second call gives the same bits."""
    from long_context_hierarchical_b200 import lh
    lens = [(37 * i) % 300 for i in range(150)]
    c = Case(lens, 4, 64, 32, "bf16", seed=9)
    q = normal(c.g, (150, 8, 1, 64), "bf16")
    o, lse = lh.decode(c.cache, c.table, c.lengths, q)
    check_decode(c, q, o, lse)
    for _ in range(3):
        o2, lse2 = lh.decode(c.cache, c.table, c.lengths, q)
        assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_decode_large_scores_and_scales(dtype):
    """One key far above the others, late and early; negative and zero scales."""
    from long_context_hierarchical_b200 import lh
    c = Case([600, 600], 1, 64, 64, dtype, seed=2)
    q = normal(c.g, (2, 2, 1, 64), dtype)
    for b, j in ((0, 590), (1, 3)):
        p = int(c.table[b, j // 64])
        c.k[p, 0, j % 64] = (q[b, 0, 0].float() * 40).to(DT[dtype])
    for scale in (None, 1.0, -0.3, 0.0):
        o, lse = lh.decode(c.cache, c.table, c.lengths, q, scale=scale)
        check_decode(c, q, o, lse, scale=scale)


def test_decode_strided_queries():
    from long_context_hierarchical_b200 import lh
    c = Case([100, 50], 2, 64, 16, "bf16")
    fused = normal(c.g, (2, 1, 12, 64), "bf16")        # [B, T, heads, d]
    q = fused[:, :, 3:7].transpose(1, 2)
    a = lh.decode(c.cache, c.table, c.lengths, q)
    b = lh.decode(c.cache, c.table, c.lengths, q.contiguous())
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    wide = torch.full((2, 40), 10 ** 9, dtype=torch.int32, device="cuda")   # a table of another stride
    wide[:, : c.width] = c.table
    a = lh.decode(c.cache, wide[:, : c.width], c.lengths, q)
    assert torch.equal(a[0], b[0])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_decode_shows_a_nan_and_survives_an_overflow(dtype):
    """A NaN in a row that is attended to reaches the head's output, and no other
    head's; scores that overflow to -inf weigh nothing (the first keys among
    them, where no finite score has been met yet)."""
    from long_context_hierarchical_b200 import lh
    c = Case([200, 200], 2, 64, 64, dtype, seed=4)
    q = normal(c.g, (2, 4, 1, 64), dtype)
    want = lh.decode(c.cache, c.table, c.lengths, q)
    c.k[int(c.table[0, 1]), 1, 5, 7] = float("nan")
    o, lse = lh.decode(c.cache, c.table, c.lengths, q)
    assert torch.isnan(lse[0, 2:]).all() and torch.isnan(o[0, 2:]).all()
    assert torch.equal(o[0, :2], want[0][0, :2]) and torch.equal(o[1], want[0][1])
    q = torch.zeros_like(q)
    q[..., 0] = 2.0
    c.k[int(c.table[0, 0])] = 0.0
    c.k[int(c.table[0, 0]), :, :17, 0] = -3e38
    ones = torch.tensor([40, 40], dtype=torch.int32, device="cuda")
    o, lse = lh.decode(c.cache, c.table, ones, q, scale=1e3)
    for h in range(4):
        assert abs(lse[0, h, 0].item() - math.log(23)) <= 2.0 ** -20
        mean = np64(c.rows(c.v, 0))[h // 2, 17:40].mean(0)
        assert np.abs(np64(o[0, h, 0]) - mean).max() <= 2.0 ** -7 * np.abs(np64(c.rows(c.v, 0))[h // 2, 17:40]).max()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rows_outside_the_cache_are_left_out_and_reported(dtype):
    from long_context_hierarchical_b200 import lh
    c = Case([100, 40], 2, 64, 16, dtype, seed=5)
    q = normal(c.g, (2, 2, 1, 64), dtype)
    lh.device_status()
    good = c.table.clone()
    bad = c.table.clone()
    bad[0, 1], bad[0, 4] = -1, c.cache.pages
    w, out = torch.zeros((2, 2, c.capacity), device="cuda"), torch.zeros((2, 2, c.capacity), device="cuda")
    o, lse = lh.decode(c.cache, bad, c.lengths, q, weights=w, weights_out=out)
    check_decode(c, q, o, lse, weights=w, weights_out=out, bad={(0, 1), (0, 4)})
    assert not out[0, :, 16:32].any()
    with pytest.raises(lh.LighthouseError) as e:
        lh.device_status()
    assert e.value.status == lh.LH_ERR_PAGE
    lh.device_status()
    # a length beyond the table and a negative one are clamped
    c.table = good
    o, lse = lh.decode(c.cache, c.table, torch.tensor([-3, 10 ** 9], dtype=torch.int32, device="cuda"), q)
    assert not o[0].any() and torch.isneginf(lse[0]).all()
    with pytest.raises(lh.LighthouseError):
        lh.device_status()
    # all pages bad: an empty sequence
    o, lse = lh.decode(c.cache, torch.full_like(good, -7), c.lengths, q)
    assert not o.any() and torch.isneginf(lse).all()
    with pytest.raises(lh.LighthouseError):
        lh.device_status()
    # append: rows whose slot or page is outside are not written
    k0, v0 = c.k.clone(), c.v.clone()
    new = normal(c.g, (2, 2, 3, 64), dtype)
    lens = torch.tensor([2, 10 ** 6], dtype=torch.int32, device="cuda")   # slots -1, 0, 1 and far behind
    t2 = good.clone()
    t2[0, 0] = c.cache.pages + 5
    lh.cache_append(c.cache, t2, lens, new, new)
    assert torch.equal(c.k.nan_to_num(9.0), k0.nan_to_num(9.0)) and torch.equal(c.v.nan_to_num(9.0), v0.nan_to_num(9.0))
    with pytest.raises(lh.LighthouseError):
        lh.device_status()
    lh.cache_append(c.cache, good, c.lengths, new, new, counts=torch.tensor([4, -1], dtype=torch.int32, device="cuda"))
    assert torch.equal(c.k.nan_to_num(9.0), k0.nan_to_num(9.0))
    with pytest.raises(lh.LighthouseError):
        lh.device_status()
    lh.device_status()


@pytest.mark.parametrize("dtype,d,layout", [("bf16", 64, "half"), ("f32", 64, "interleaved"), ("bf16", 128, "half"),
                                            ("f32", 128, "half")])
@pytest.mark.parametrize("B,T,G,page", [(1, 1, 1, 16), (5, 1, 4, 32), (3, 70, 2, 16), (2, 129, 1, 64)])
def test_append(dtype, d, layout, B, T, G, page):
    from long_context_hierarchical_b200 import lh
    H = 2
    lens = [T + 5 * b for b in range(B)]
    c = Case(lens, H, d, page, dtype, seed=T)
    k0, v0 = c.k.clone(), c.v.clone()
    q = normal(c.g, (B, T, H * G, d), dtype).transpose(1, 2)
    k, v = (normal(c.g, (B, T, H, d), dtype).transpose(1, 2) for _ in range(2))
    rp = lh.rotary_plan(d, layout=layout)
    f = oracle.frequencies(d)
    counts = torch.tensor([(T - 3 * b) if T > 3 * b else 0 for b in range(B)], dtype=torch.int32, device="cuda")
    sp = torch.full((B, H, c.capacity), -9, dtype=torch.int32, device="cuda")
    pos = torch.randint(0, 10000, (B, T), generator=c.g, device="cuda", dtype=torch.int32)
    for positions, cnt in ((None, None), (pos, counts)):
        c.k.copy_(k0)
        c.v.copy_(v0)
        sp.fill_(-9)
        qo = lh.cache_append(c.cache, c.table, c.lengths, k, v, Q=q, rotary=rp, positions=positions, counts=cnt,
                             slot_positions=sp)
        want_k, want_v = k0.clone(), v0.clone()
        for b, n in enumerate(lens):
            m = T if cnt is None else int(cnt[b])
            slots = np.arange(n - m, n)
            p = slots if positions is None else np64(positions[b, :m])
            if m:
                check_rotary(qo[b: b + 1, :, :m], q[b: b + 1, :, :m], p[None], f, layout)
            assert not qo[b, :, m:].any()
            ids = c.table[b].long()[torch.from_numpy(slots // page).cuda()]
            rows = torch.from_numpy(slots % page).cuda()
            if m:
                got = c.k[ids, :, rows].transpose(0, 1)[None]
                check_rotary(got, k[b: b + 1, :, :m], p[None], f, layout)
                want_k[ids, :, rows] = c.k[ids, :, rows]
                want_v[ids, :, rows] = v[b, :, :m].transpose(0, 1)
                want = torch.full((H, c.capacity), -9, dtype=torch.int32, device="cuda")
                want[:, n - m: n] = torch.as_tensor(p, device="cuda").int()
                assert torch.equal(sp[b], want)
        assert torch.equal(c.k.nan_to_num(9.0), want_k.nan_to_num(9.0))   # nothing else was written
        assert torch.equal(c.v.nan_to_num(9.0), want_v.nan_to_num(9.0))
    # without rotary: copies; no queries: no answer
    assert lh.cache_append(c.cache, c.table, c.lengths, k, v) is None
    for b, n in enumerate(lens):
        assert torch.equal(c.rows(c.k, b)[:, n - T:], k[b]) and torch.equal(c.rows(c.v, b)[:, n - T:], v[b])
    # queries in place
    q2 = q.clone()
    want = lh.cache_append(c.cache, c.table, c.lengths, k, v, Q=q, rotary=rp)
    assert torch.equal(lh.cache_append(c.cache, c.table, c.lengths, k, v, Q=q2, rotary=rp, out=q2), want)
    lh.device_status()


# --- eviction ----------------------------------------------------------------------------


def check_evict(c, weights, budget, got, k0, v0, positions=None, protect=None):
    n_out, w_out, p_out = got
    want_k, want_v = k0.clone(), v0.clone()
    for b, n in enumerate(c.lens):
        m = min(n, budget)
        assert int(n_out[b]) == m
        for h in range(c.H):
            pos = None if positions is None else positions[b, h].cpu().numpy()
            _, moves, _ = oracle.evict(weights[b, h].cpu().numpy(), n, budget, pos,
                                       None if protect is None else int(protect[b]))
            w = torch.zeros(c.capacity, device="cuda")
            w[:m] = weights[b, h, :m]
            p = torch.full((c.capacity,), -1, dtype=torch.int32, device="cuda")
            if positions is not None:
                p[:m] = positions[b, h, :m]
            if moves:
                src, dst = (torch.tensor(x, device="cuda") for x in zip(*moves))
                ps, pd = c.table[b].long()[src // c.page], c.table[b].long()[dst // c.page]
                want_k[pd, h, dst % c.page] = k0[ps, h, src % c.page]
                want_v[pd, h, dst % c.page] = v0[ps, h, src % c.page]
                w[dst] = weights[b, h, src]
                if positions is not None:
                    p[dst] = positions[b, h, src]
            assert torch.equal(w_out[b, h].nan_to_num(-1.0), w.nan_to_num(-1.0)), (b, h)
            if positions is not None:
                assert torch.equal(p_out[b, h], p), (b, h)
    assert (p_out is None) == (positions is None)
    assert torch.equal(c.k.nan_to_num(9.0), want_k.nan_to_num(9.0))
    assert torch.equal(c.v.nan_to_num(9.0), want_v.nan_to_num(9.0))


def make_weights(c, kind):
    shape = (len(c.lens), c.H, c.capacity)
    if kind == "ties":
        return torch.randint(0, 3, shape, generator=c.g, device="cuda").float()
    if kind == "equal":
        return torch.ones(shape, device="cuda")
    w = torch.exp(3.0 * torch.randn(shape, generator=c.g, device="cuda"))
    if kind == "odd":   # signs, zeros of both signs, infinities, NaN, denormals
        special = torch.tensor([0.0, -0.0, math.inf, -math.inf, math.nan, 1e-42, -1e-42, -3.0], device="cuda")
        at = torch.randint(0, 16, shape, generator=c.g, device="cuda")
        w = torch.where(at < 8, special[at.clamp(max=7)], w)
    return w


@pytest.mark.parametrize("dtype,d", [("bf16", 64), ("f32", 64), ("bf16", 128), ("f32", 128)])
@pytest.mark.parametrize("kind", ["spread", "ties", "equal", "odd"])
@pytest.mark.parametrize("lens,budget", [([1, 0, 2], 1), ([100, 37, 64, 65], 64), ([5000, 4097, 4096, 1], 4096),
                                         ([9001], 13), ([300], 299), ([40, 50], 1000)])
def test_evict(dtype, d, kind, lens, budget):
    from long_context_hierarchical_b200 import lh
    c = Case(lens, 2, d, 16, dtype, seed=budget, width=-(-max(lens) // 16) + 1)
    w = make_weights(c, kind)
    for b, n in enumerate(lens):
        w[b, :, n:] = 0.0
    k0, v0 = c.k.clone(), c.v.clone()
    check_evict(c, w, budget, lh.evict(c.cache, c.table, c.lengths, w, budget), k0, v0)
    lh.device_status()


@pytest.mark.parametrize("kind", ["spread", "ties"])
@pytest.mark.parametrize("recent", [0, 1, 30, 64, 90])
def test_evict_protected_rows_and_positions(kind, recent):
    from long_context_hierarchical_b200 import lh
    lens, budget = [200, 100, 64, 3, 0], 64
    c = Case(lens, 3, 64, 32, "bf16", seed=recent)
    w = make_weights(c, kind)
    pos = torch.rand(w.shape, generator=c.g, device="cuda").argsort(-1).int()
    protect = torch.tensor([c.capacity - recent] * 5, dtype=torch.int32, device="cuda")
    k0, v0 = c.k.clone(), c.v.clone()
    got = lh.evict(c.cache, c.table, c.lengths, w, budget, positions=pos, protect=protect)
    check_evict(c, w, budget, got, k0, v0, pos, protect)
    # in place, from the same start
    c.k.copy_(k0)
    c.v.copy_(v0)
    w2, p2 = w.clone(), pos.clone()
    again = lh.evict(c.cache, c.table, c.lengths, w2, budget, positions=p2, protect=protect, weights_out=w2,
                     positions_out=p2)
    assert again[1] is w2 and torch.equal(w2, got[1]) and torch.equal(p2, got[2]) and torch.equal(again[0], got[0])
    check_evict(c, w, budget, again, k0, v0, pos, protect)
    # chronological slots: the last rows of each sequence
    c.k.copy_(k0)
    c.v.copy_(v0)
    protect = (c.lengths - recent).int()
    check_evict(c, w, budget, lh.evict(c.cache, c.table, c.lengths, w, budget, protect=protect), k0, v0, None, protect)


def test_evict_long():
    from long_context_hierarchical_b200 import lh
    c = Case([98304 + 5], 2, 64, 64, "bf16", seed=1)
    for kind in ("spread", "ties"):
        w = make_weights(c, kind)
        w[:, :, c.lens[0]:] = 0.0
        k0, v0 = c.k.clone(), c.v.clone()
        check_evict(c, w, 49152, lh.evict(c.cache, c.table, c.lengths, w, 49152), k0, v0)


@pytest.mark.parametrize("kind", ["spread", "ties", "equal"])
@pytest.mark.parametrize("H,n", [(26, 6100), (20, 6101), (14, 6102), (10, 8103), (8, 10104), (6, 12105), (1, 14106),
                                 (5, 16507)])
def test_evict_heads_of_one_to_eight_blocks(H, n, kind):
    # three sequences of H heads: from many heads of one block to few of eight; the
    # shorter sequences leave some blocks of a head without a slot
    from long_context_hierarchical_b200 import lh
    c = Case([n, 5, n // 2], H, 64, 16, "bf16", seed=n)
    w = make_weights(c, kind)
    protect = (c.lengths - 300).int()
    for budget in (n // 3, n - 40):
        k0, v0 = c.k.clone(), c.v.clone()
        check_evict(c, w, budget, lh.evict(c.cache, c.table, c.lengths, w, budget, protect=protect), k0, v0, None,
                    protect)
        c.k.copy_(k0)
        c.v.copy_(v0)
    lh.device_status()


@pytest.mark.parametrize("protected", [False, True])
@pytest.mark.parametrize("placed", [False, True])
@pytest.mark.parametrize("in_place", [False, True])
def test_evict_more_slots_than_a_block_holds(protected, placed, in_place):
    """Many heads of more slots than the selection keeps in shared memory: it
    reads the weights again in each pass."""
    from long_context_hierarchical_b200 import lh
    n, H, budget, page = 41003, 64, 20000, 128
    c = Case([n], H, 64, page, "bf16", seed=6)
    w = make_weights(c, "ties" if protected else "spread")
    w[:, :, n:] = 0.0
    pos = torch.rand(w.shape, generator=c.g, device="cuda").argsort(-1).int() if placed else None
    protect = torch.tensor([30000], dtype=torch.int32, device="cuda") if protected else None
    k0, v0 = c.k.clone(), c.v.clone()
    w0, p0 = w.clone(), None if pos is None else pos.clone()
    got = lh.evict(c.cache, c.table, c.lengths, w, budget, positions=pos, protect=protect,
                   weights_out=w if in_place else None, positions_out=pos if in_place else None)
    assert int(got[0][0]) == budget
    for h in (0, 17, 63):
        _, moves, _ = oracle.evict(w0[0, h].cpu().numpy(), n, budget, None if p0 is None else p0[0, h].cpu().numpy(),
                                   None if protect is None else 30000)
        src, dst = (torch.tensor(x, device="cuda") for x in zip(*moves))
        want = torch.zeros(c.capacity, device="cuda")
        want[:budget] = w0[0, h, :budget]
        want[dst] = w0[0, h, src]
        assert torch.equal(got[1][0, h], want)
        if placed:
            p = torch.full((c.capacity,), -1, dtype=torch.int32, device="cuda")
            p[:budget] = p0[0, h, :budget]
            p[dst] = p0[0, h, src]
            assert torch.equal(got[2][0, h], p)
        table = c.table[0].long()
        for x, x0 in ((c.k, k0), (c.v, v0)):
            rows = x0[:, h].clone()
            rows[table[dst // page], dst % page] = x0[table[src // page], h, src % page]
            assert torch.equal(x[:, h].nan_to_num(9.0), rows.nan_to_num(9.0))


def test_evict_bad_pages_move_no_rows():
    from long_context_hierarchical_b200 import lh
    c = Case([64], 1, 64, 16, "bf16")
    w = torch.arange(64, device="cuda", dtype=torch.float32).view(1, 1, 64)
    k0, v0 = c.k.clone(), c.v.clone()
    lh.device_status()
    bad = c.table.clone()
    bad[0, 3] = -1
    n, wo, _ = lh.evict(c.cache, bad, c.lengths, w, 16)
    assert int(n[0]) == 16 and torch.equal(wo[0, 0, :16].sort().values, w[0, 0, 48:])
    assert torch.equal(c.k.nan_to_num(9.0), k0.nan_to_num(9.0)) and torch.equal(c.v.nan_to_num(9.0), v0.nan_to_num(9.0))
    with pytest.raises(lh.LighthouseError) as e:
        lh.device_status()
    assert e.value.status == lh.LH_ERR_PAGE


# --- together ------------------------------------------------------------------------------


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_answering_with_a_short_cache(dtype):
    """Prompt, then steps of append, attention with weights and eviction, against
    plain lists of rows; what is kept is taken from the GPU's own weights, so
    the two sides cannot part at a near tie."""
    from long_context_hierarchical_b200 import lh
    B, H, Hq, d, page, budget, recent = 2, 2, 4, 64, 16, 48, 8
    g = gen(12)
    rp = lh.rotary_plan(d)
    f = oracle.frequencies(d)
    width = 5
    kc = lh.PagedCache(B * width, page, H, d, dtype)
    table = torch.arange(B * width, dtype=torch.int32, device="cuda").view(B, width)
    lengths = torch.zeros(B, dtype=torch.int32, device="cuda")
    cap = width * page
    weights = torch.zeros((B, H, cap), device="cuda")
    positions = torch.full((B, H, cap), -1, dtype=torch.int32, device="cuda")
    held = [[{} for _ in range(H)] for _ in range(B)]   # position -> (k, v) as stored
    at = torch.zeros(B, dtype=torch.int32, device="cuda")
    for step, T in enumerate([40, 1, 1, 20, 1, 1, 1, 1]):
        k, v = normal(g, (B, H, T, d), dtype), normal(g, (B, H, T, d), dtype)
        q = normal(g, (B, Hq, T, d), dtype)
        lengths += T
        pos = (at[:, None] + torch.arange(T, device="cuda", dtype=torch.int32)).int()
        at += T
        qr = lh.cache_append(kc, table, lengths, k, v, Q=q, rotary=rp, positions=pos, slot_positions=positions)
        last = qr[:, :, -1:]
        check_rotary(last, q[:, :, -1:], np64(pos[:, -1:]), f, "half")
        kt = lh.rotary(rp, k, positions=pos)
        for b in range(B):
            for h in range(H):
                for t in range(T):
                    held[b][h][int(pos[b, t])] = (kt[b, h, t], v[b, h, t])
        before = weights.clone()
        o, lse = lh.decode(kc, table, lengths, last, weights=weights)
        for b in range(B):
            n = int(lengths[b])
            for h in range(H):
                order = positions[b, h, :n].tolist()
                assert sorted(order) == sorted(held[b][h])
                kk = np.stack([np64(held[b][h][p][0]) for p in order])[None]
                vv = np.stack([np64(held[b][h][p][1]) for p in order])[None]
                qq = np64(last[b, h * 2: h * 2 + 2, 0])
                wo, wl, p = oracle.decode(qq, kk, vv, d ** -0.5)
                tol = 2.0 ** -6 if dtype == "bf16" else 2.0 ** -16
                T_o = np.einsum("hn,nd->hd", p, np.abs(vv[0]))
                assert np.all(np.abs(np64(o[b, h * 2: h * 2 + 2, 0]) - wo) <= tol * (T_o + np.abs(wo)))
                grew = np64(weights[b, h, :n] - before[b, h, :n])
                assert np.abs(grew - p.sum(0)).max() <= 2.0 ** -14
        protect = (at - recent).int()
        new_len, weights, positions = lh.evict(kc, table, lengths, weights, budget, positions=positions,
                                               protect=protect)
        for b in range(B):
            for h in range(H):
                left = positions[b, h, : int(new_len[b])].tolist()
                assert len(set(left)) == len(left) == min(int(lengths[b]), budget)
                assert all(p in left for p in held[b][h] if p >= int(protect[b]))
                held[b][h] = {p: held[b][h][p] for p in left}
        lengths = new_len
    lh.device_status()


def test_training_then_answering_on_the_same_rows():
    """Dense attention's last row over rotated Q and K is what decoding gives over a cache
    filled with the same rows: within a rounding of each side's own bound (2^-6 of T)."""
    from long_context_hierarchical_b200 import lh
    B, H, N, d = 2, 2, 200, 64
    g = gen(13)
    q, k, v = (normal(g, (B, H, N, d), "bf16") for _ in range(3))
    rp = lh.rotary_plan(d)
    qr, kr = lh.rotary(rp, q, k)
    O, lse = lh.attn_fwd(qr, kr, v)
    kc = lh.PagedCache(B * 13, 16, H, d)
    table = torch.randperm(B * 13, generator=g, device="cuda", dtype=torch.int32).view(B, 13)
    lengths = torch.full((B,), N, dtype=torch.int32, device="cuda")
    qa = lh.cache_append(kc, table, lengths, k, v, Q=q, rotary=rp)
    assert torch.equal(qa, qr)
    o, l1 = lh.decode(kc, table, lengths, qa[:, :, -1:])
    scale = np64(v).__abs__().max()
    assert np.abs(np64(o[:, :, 0]) - np64(O[:, :, -1])).max() <= 2.0 ** -6 * scale
    assert np.abs(np64(l1[:, :, 0]) - np64(lse[:, :, -1])).max() <= 2.0 ** -10


# --- graphs and streams -----------------------------------------------------------------------


def test_step_in_a_captured_graph_follows_its_inputs():
    """A step captured at one length is right at later ones: lengths, tables and
    inputs are read when the graph runs."""
    from long_context_hierarchical_b200 import lh
    c = Case([90, 3], 2, 64, 16, "bf16", seed=3, width=8)
    full = torch.randperm(16, device="cuda", dtype=torch.int32)
    k = torch.zeros((16, 2, 16, 64), device="cuda", dtype=torch.bfloat16)
    v = k.clone()
    kc = lh.PagedCache.of(k, v)
    table = full.view(2, 8).contiguous()
    lengths = torch.tensor([90, 3], dtype=torch.int32, device="cuda")
    k.copy_(normal(c.g, k.shape, "bf16"))
    v.copy_(normal(c.g, v.shape, "bf16"))
    rp = lh.rotary_plan(64)
    nk, nv, nq = (normal(c.g, (2, h, 1, 64), "bf16") for h in (2, 2, 4))
    weights = torch.zeros((2, 2, 128), device="cuda")

    def step():
        lengths.add_(1)
        q = lh.cache_append(kc, table, lengths, nk, nv, Q=nq, rotary=rp)
        o, lse = lh.decode(kc, table, lengths, q, weights=weights)
        n, w, _ = lh.evict(kc, table, lengths, weights, 64)
        return q, o, lse, n, w

    held = (k, v, lengths, weights, nk)
    start = [t.clone() for t in held]

    def reset():
        for t, s in zip(held, start):
            t.copy_(s)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    reset()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    reset()
    eager = []
    for i in range(3):
        nk.add_(0.5)
        eager.append([t.clone() for t in step()] + [k.clone(), v.clone(), weights.clone()])
    reset()
    for i in range(3):
        nk.add_(0.5)
        graph.replay()
        for a, b in zip((*outs, k, v, weights), eager[i]):
            assert torch.equal(a, b), i
    torch.cuda.synchronize()
    lh.device_status()


def test_calls_on_another_stream_and_two_at_once():
    from long_context_hierarchical_b200 import lh
    c = Case([3000, 1200], 4, 64, 64, "bf16", seed=8)
    q = normal(c.g, (2, 8, 1, 64), "bf16")
    want = lh.decode(c.cache, c.table, c.lengths, q)
    rp = lh.rotary_plan(64)
    x = normal(c.g, (2, 4, 999, 64), "bf16")
    turned = lh.rotary(rp, x)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    got = []
    for i in range(24):
        s = streams[i % 3]
        got.append(lh.decode(c.cache, c.table, c.lengths, q, stream=s))
        got.append((lh.rotary(rp, x, stream=s),))
        torch.empty(1 << 20, device="cuda").fill_(float(i))   # memory of the current stream
    torch.cuda.synchronize()
    for i, g in enumerate(got):
        for a, b in zip(g, want if i % 2 == 0 else (turned,)):
            assert torch.equal(a, b)
    with pytest.raises((ValueError, RuntimeError)):
        lh.rotary(rp, x.cpu())


def test_append_and_evict_on_another_stream():
    from long_context_hierarchical_b200 import lh
    rp = lh.rotary_plan(64)
    sides = []
    for other in (False, True):
        c = Case([300, 90], 2, 64, 16, "bf16", seed=31)
        new = normal(c.g, (2, 2, 20, 64), "bf16")
        w = make_weights(c, "spread")
        stream = torch.cuda.Stream() if other else None
        torch.cuda.synchronize()
        q = lh.cache_append(c.cache, c.table, c.lengths, new, new, Q=new, rotary=rp, stream=stream)
        got = lh.evict(c.cache, c.table, c.lengths, w, 64, stream=stream)
        junk = [torch.full((1 << 16,), float(i), device="cuda") for i in range(8)]   # the current stream goes on
        torch.cuda.synchronize()
        del junk
        sides.append((q, got[0], got[1], c.k.nan_to_num(9.0), c.v.nan_to_num(9.0)))
    for a, b in zip(*sides):
        assert torch.equal(a, b)


def test_two_captured_graphs_at_once():
    """Each capture has its own workspace, so two graphs may run side by side."""
    from long_context_hierarchical_b200 import lh
    cases = [Case([5000, 700], 2, 64, 64, "bf16", seed=40 + i) for i in range(2)]
    qs = [normal(c.g, (2, 4, 1, 64), "bf16") for c in cases]
    ws = [make_weights(c, "spread") for c in cases]
    want = [lh.decode(c.cache, c.table, c.lengths, q) for c, q in zip(cases, qs)]
    cut = [lh.evict(lh.PagedCache.of(c.k.clone(), c.v.clone()), c.table, c.lengths, w, 600)[1]
           for c, w in zip(cases, ws)]
    graphs, outs, keep = [], [], []
    for c, q, w in zip(cases, qs, ws):
        copy = lh.PagedCache.of(c.k.clone(), c.v.clone())
        keep.append(copy)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append((*lh.decode(c.cache, c.table, c.lengths, q),
                         lh.evict(copy, c.table, c.lengths, w, 600)[1]))
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(10):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for o, w, e in zip(outs, want, cut):
        assert torch.equal(o[0], w[0]) and torch.equal(o[1], w[1]) and torch.equal(o[2], e)


def test_calls_without_rows():
    from long_context_hierarchical_b200 import lh
    c = Case([20, 0], 2, 64, 16, "bf16")
    k0 = c.k.clone()
    none = torch.zeros((2, 2, 0, 64), dtype=torch.bfloat16, device="cuda")
    assert lh.cache_append(c.cache, c.table, c.lengths, none, none, Q=none, rotary=lh.rotary_plan(64)).shape == none.shape
    zero = torch.zeros(2, dtype=torch.int32, device="cuda")
    one = normal(c.g, (2, 2, 1, 64), "bf16")
    q = lh.cache_append(c.cache, c.table, c.lengths, one, one, Q=one, counts=zero)
    assert not q.any() and torch.equal(c.k.nan_to_num(9.0), k0.nan_to_num(9.0))
    empty = torch.zeros((0, 3), dtype=torch.int32, device="cuda")
    o, lse = lh.decode(c.cache, empty, zero[:0], one[:0, :, :, :])
    assert o.shape == (0, 2, 1, 64) and lse.shape == (0, 2, 1)
    n, w, p = lh.evict(c.cache, empty, zero[:0], torch.zeros((0, 2, 48), device="cuda"), 5)
    assert n.shape == (0,) and w.shape == (0, 2, 48) and p is None
    lh.device_status()


def test_tensors_of_a_device_that_is_not_current():
    from long_context_hierarchical_b200 import lh
    if torch.cuda.device_count() < 2:
        pytest.skip("one GPU")
    rp = lh.rotary_plan(64)
    x = torch.randn(1, 2, 70, 64, device="cuda:1")
    got = lh.rotary(rp, x)
    assert got.device == x.device and torch.equal(got.cpu(), lh.rotary(rp, x.to("cuda:0")).cpu())
    with pytest.raises(ValueError):
        lh.rotary(rp, x, x.to("cuda:0"))
    with pytest.raises(ValueError):
        lh.rotary(rp, x, stream=torch.cuda.Stream("cuda:0"))


def test_offsets_past_32_bits():
    """A cache of more than 2^31 elements: rows at its far end are found."""
    from long_context_hierarchical_b200 import lh
    page, d = 1024, 128
    pages = (1 << 31) // (page * d) + 8
    k = torch.zeros((pages, 1, page, d), dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    kc = lh.PagedCache.of(k, v)
    g = gen(20)
    n = 1500
    table = torch.tensor([[pages - 1, pages - 5]], dtype=torch.int32, device="cuda")
    lengths = torch.tensor([n], dtype=torch.int32, device="cuda")
    nk, nv = normal(g, (1, 1, n, d), "bf16"), normal(g, (1, 1, n, d), "bf16")
    lh.cache_append(kc, table, lengths, nk, nv)
    assert torch.equal(k[pages - 1, 0], nk[0, 0, :page]) and torch.equal(v[pages - 5, 0, : n - page], nv[0, 0, page:])
    c = Case.__new__(Case)
    c.k, c.v, c.table, c.lengths, c.lens = k, v, table, lengths, [n]
    c.H, c.d, c.page, c.dtype, c.width = 1, d, page, "bf16", 2
    c.cache, c.capacity, c.g = kc, 2 * page, g
    q = normal(g, (1, 2, 1, d), "bf16")
    check_decode(c, q, *lh.decode(kc, table, lengths, q))
    w = torch.rand((1, 1, 2 * page), generator=g, device="cuda")
    w[..., n:] = 0.0
    new = lh.evict(kc, table, lengths, w, 700)
    _, moves, _ = oracle.evict(w[0, 0].cpu().numpy(), n, 700)
    src, dst = (torch.tensor(x) for x in zip(*moves))
    assert torch.equal(k[pages - 1, 0].cpu()[dst], nk[0, 0].cpu()[src])
    assert int(new[0]) == 700
    lh.device_status()
