"""Rotary positions and paged cache without a GPU: the oracle's pins, and the
refusals of the library and its binding (nothing here launches a kernel)."""
import ctypes
import math

import numpy as np
import pytest
import torch

from long_context_hierarchical_b200 import lh
from oracle import cache as oracle

# --- the oracle -----------------------------------------------------------------


def test_oracle_rotation_is_a_complex_product():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((3, 5, 64))
    pos = np.array([0, 1, 7, 1000, -3])
    for layout in ("half", "interleaved"):
        f = oracle.frequencies(32)
        y = oracle.rotate(x, pos, f, layout, 1.5)
        a = x[..., :16] + 1j * x[..., 16:32] if layout == "half" else x[..., 0:32:2] + 1j * x[..., 1:32:2]
        z = 1.5 * a * np.exp(1j * pos[:, None] * f)
        got = y[..., :16] + 1j * y[..., 16:32] if layout == "half" else y[..., 0:32:2] + 1j * y[..., 1:32:2]
        assert np.abs(got - z).max() < 1e-12
        assert np.array_equal(y[..., 32:], x[..., 32:])
        # the transposed map is the adjoint: <g, R x> = <R' g, x>
        g = rng.standard_normal(x.shape)
        back = oracle.rotate(g, pos, f, layout, 1.5, transpose=True)
        assert abs((g * y).sum() - (back * x).sum()) < 1e-9


def test_oracle_rotated_products_depend_on_the_distance_alone():
    rng = np.random.default_rng(1)
    q, k = rng.standard_normal((2, 64))
    f = oracle.frequencies(64)
    dot = [oracle.rotate(q[None], [t + 5], f, "half")[0] @ oracle.rotate(k[None], [t], f, "half")[0]
           for t in (0, 11, 4000)]
    assert max(dot) - min(dot) < 1e-9


def test_oracle_frequencies_by_hand():
    f = oracle.frequencies(4, base=100.0)
    assert np.allclose(f, [1.0, 0.1])
    assert np.allclose(oracle.frequencies(4, base=100.0, scaling="linear", factor=4.0), [0.25, 0.025])
    # 2 pi * 10 positions: 10 turns and 1 turn; ramp from 1 to 4 turns
    b = oracle.frequencies(4, base=100.0, scaling="bands", factor=8.0, low=1.0, high=4.0, original=20 * math.pi)
    assert np.allclose(b, [1.0, 0.1 / 8.0])
    b = oracle.frequencies(4, base=100.0, scaling="bands", factor=8.0, low=0.0, high=4.0, original=20 * math.pi)
    assert np.allclose(b[1], 0.75 * 0.1 / 8.0 + 0.25 * 0.1)


def test_oracle_decode_by_hand():
    k = np.array([[[1.0, 0.0], [0.0, 1.0]]])
    v = np.array([[[2.0, 0.0], [0.0, 4.0]]])
    q = np.array([[math.log(3.0), 0.0], [0.0, 0.0]])
    o, lse, p = oracle.decode(q, k, v, 1.0)
    assert np.allclose(p, [[0.75, 0.25], [0.5, 0.5]])
    assert np.allclose(o, [[1.5, 1.0], [1.0, 2.0]])
    assert np.allclose(lse, [math.log(4.0), math.log(2.0)])
    o, lse, p = oracle.decode(q, k[:, :0], v[:, :0], 1.0)
    assert not o.any() and np.isneginf(lse).all()


@pytest.mark.parametrize("kw,m,moves", [
    (dict(weights=[5, 1, 4, 2, 3], n=5, budget=3), 3, [(4, 1)]),
    (dict(weights=[1, 1, 1, 1], n=4, budget=2), 2, []),                       # ties: the lower slots
    (dict(weights=[0, 0, 9, 8, 7], n=5, budget=3), 3, [(3, 0), (4, 1)]),
    (dict(weights=[5, 1, 4, 2, 3], n=5, budget=3, protect=3), 3, [(3, 1), (4, 2)]),
    (dict(weights=[5, 1, 4, 2, 3], n=5, budget=2, protect=1), 2, [(2, 0), (4, 1)]),  # more protected than budget
    (dict(weights=[5, float("nan"), 0, 2], n=4, budget=3), 3, [(3, 1)]),
    (dict(weights=[5, 1, 4], n=3, budget=8), 3, []),
    (dict(weights=[5, 1, 4, 2], n=4, budget=2, positions=[3, 2, 1, 0], protect=2), 2, []),
    (dict(weights=[], n=0, budget=2), 0, []),
])
def test_oracle_eviction_by_hand(kw, m, moves):
    got = oracle.evict(**kw)
    assert got[:2] == (m, moves)
    assert len(got[2]) == m


# --- the plan ---------------------------------------------------------------------


@pytest.mark.parametrize("kw", [
    dict(d=64), dict(d=128, rot=32, base=500000.0),
    dict(d=64, scaling="linear", factor=4.0),
    dict(d=128, scaling="bands", factor=8.0, low=1.0, high=4.0, original=8192),
    dict(d=64, rot=16, layout="interleaved", scaling="linear", factor=0.5, base=1e-3),
])
def test_rotary_plan_frequencies_match_the_oracle(kw):
    rp = lh.rotary_plan(**kw)
    rot = kw.get("rot", kw["d"])
    f = oracle.frequencies(rot, **{k: v for k, v in kw.items() if k not in ("d", "rot", "layout")})
    turns = np.array(list(rp.raw.turns), dtype=np.float64) / 2.0 ** 64
    # one fp64 step of the power, the division and the product each: 2^-50 of the turns
    want = f / (2 * math.pi)
    off = np.abs(turns[: rot // 2] - (want - np.floor(want)))
    assert np.all(np.minimum(off, 1.0 - off) <= 2.0 ** -50 * np.maximum(want, 2.0 ** -10))
    assert not turns[rot // 2:].any()


@pytest.mark.parametrize("kw,status", [
    (dict(d=96), lh.LH_ERR_UNSUPPORTED),
    (dict(d=64, rot=24), lh.LH_ERR_UNSUPPORTED),
    (dict(d=64, rot=80), lh.LH_ERR_INVALID_ARG),
    (dict(d=64, rot=0), lh.LH_ERR_INVALID_ARG),
    (dict(base=0.0), lh.LH_ERR_INVALID_ARG),
    (dict(base=float("nan")), lh.LH_ERR_INVALID_ARG),
    (dict(base=1e-300, d=128, scaling="linear", factor=1e-300), lh.LH_ERR_INVALID_ARG),
    (dict(magnitude=-1.0), lh.LH_ERR_INVALID_ARG),
    (dict(scaling="linear", factor=0.0), lh.LH_ERR_INVALID_ARG),
    (dict(scaling="bands", factor=8.0), lh.LH_ERR_INVALID_ARG),                          # original missing
    (dict(scaling="bands", factor=8.0, original=8192, low=4.0), lh.LH_ERR_INVALID_ARG),  # high <= low
])
def test_rotary_plan_refusals(kw, status):
    with pytest.raises(lh.LighthouseError) as e:
        lh.rotary_plan(**kw)
    assert e.value.status == status


# --- the entry points ---------------------------------------------------------------

GOOD = 1 << 20  # aligned, never dereferenced here


def rows(ptr=GOOD, H=2, sb=2 * 8 * 64, sh=8 * 64, sn=64):
    return lh.LhRows(ptr, sb, sh, sn, H)


def cache(**kw):
    c = dict(k=GOOD, v=GOOD << 4, pages=8, H=2, page=16, d=64, dtype=lh.LH_BF16, table=GOOD, table_stride=4,
             B=2, width=4, lengths=GOOD)
    c.update(kw)
    return lh.LhCache(*(c[n] for n, _ in lh.LhCache._fields_))


def call_rotary(x=None, y=None, B=2, N=8, count=1, dtype=lh.LH_BF16, positions=None, stride=0, plan=None):
    p = lh.rotary_plan(64).raw if plan is None else plan
    x = rows() if x is None else x
    y = rows(ptr=GOOD << 4) if y is None else y
    return lh.LIB.lh_rotary(ctypes.byref(p), dtype, B, N, count, ctypes.byref(x), ctypes.byref(y), positions,
                            stride, 0, 0, None)


def test_rotary_refusals():
    bad = lh.LH_ERR_INVALID_ARG
    forged = lh.LhRotaryPlan.from_buffer_copy(lh.rotary_plan(64).raw)
    forged.turns[3] += 1
    assert call_rotary(plan=forged) == bad
    assert call_rotary(dtype=7) == lh.LH_ERR_UNSUPPORTED
    assert call_rotary(N=-1) == bad and call_rotary(B=1 << 20, N=1 << 20) == bad
    assert call_rotary(count=3) == bad and call_rotary(count=0) == bad
    assert call_rotary(x=rows(ptr=GOOD + 8)) == bad and call_rotary(x=rows(ptr=None)) == bad
    assert call_rotary(x=rows(sn=68)) == bad                       # rows off the 16-byte boundary
    assert call_rotary(x=rows(sn=-64)) == bad
    assert call_rotary(x=rows(sb=1 << 58)) == bad and b"too large" in lh.LIB.lh_last_error()
    assert call_rotary(y=rows(ptr=GOOD << 4, sn=0)) == bad         # output rows on one another
    assert b"overlap" in lh.LIB.lh_last_error()
    assert call_rotary(y=rows(ptr=GOOD << 4, sh=64 * 4)) == bad
    assert call_rotary(y=rows(ptr=GOOD << 4, H=3, sb=3 * 8 * 64)) == bad   # H differs
    assert call_rotary(y=rows(ptr=GOOD + 64 * 2)) == bad           # shifted by one row: overlaps its input
    assert call_rotary(x=rows(H=0)) == bad
    assert call_rotary(positions=ctypes.c_void_p(GOOD + 2)) == bad
    assert call_rotary(positions=ctypes.c_void_p(GOOD), stride=-1) == bad
    two = (lh.LhRows * 2)(rows(), rows(ptr=GOOD << 1))
    for outs in ((GOOD << 4, GOOD << 4), (GOOD << 1, GOOD << 4), (GOOD << 4, GOOD)):  # on one another, or exchanged
        y = (lh.LhRows * 2)(*(rows(ptr=p) for p in outs))
        assert lh.LIB.lh_rotary(ctypes.byref(lh.rotary_plan(64).raw), lh.LH_BF16, 2, 8, 2, ctypes.byref(two),
                                ctypes.byref(y), None, 0, 0, 0, None) == bad
    for start in (2 ** 31 - 7, -2 ** 31 - 1):
        assert lh.LIB.lh_rotary(ctypes.byref(lh.rotary_plan(64).raw), lh.LH_BF16, 2, 8, 1, ctypes.byref(rows()),
                                ctypes.byref(rows(ptr=GOOD << 4)), None, 0, start, 0, None) == bad
    assert call_rotary(N=0) == lh.LH_OK and call_rotary(B=0) == lh.LH_OK   # nothing to do


@pytest.mark.parametrize("kw,status", [
    (dict(k=None), lh.LH_ERR_INVALID_ARG), (dict(v=GOOD + 8), lh.LH_ERR_INVALID_ARG),
    (dict(pages=0), lh.LH_ERR_INVALID_ARG), (dict(H=0), lh.LH_ERR_INVALID_ARG),
    (dict(B=0), lh.LH_ERR_INVALID_ARG), (dict(width=0), lh.LH_ERR_INVALID_ARG),
    (dict(page=8), lh.LH_ERR_UNSUPPORTED), (dict(page=48), lh.LH_ERR_UNSUPPORTED),
    (dict(page=1 << 17), lh.LH_ERR_UNSUPPORTED), (dict(d=96), lh.LH_ERR_UNSUPPORTED),
    (dict(dtype=3), lh.LH_ERR_UNSUPPORTED), (dict(table=None), lh.LH_ERR_INVALID_ARG),
    (dict(lengths=GOOD + 2), lh.LH_ERR_INVALID_ARG), (dict(table_stride=-4), lh.LH_ERR_INVALID_ARG),
    (dict(width=1 << 15, page=1 << 16), lh.LH_ERR_UNSUPPORTED),     # capacity 2^31
    (dict(B=65536, H=1), lh.LH_ERR_UNSUPPORTED),
    (dict(pages=(1 << 31) - 1, H=32767, B=2, page=65536, width=1, d=128), lh.LH_ERR_INVALID_ARG),  # 2^70 bytes
    (dict(v=GOOD), lh.LH_ERR_INVALID_ARG), (dict(v=GOOD + 4096), lh.LH_ERR_INVALID_ARG),   # on one another
])
def test_cache_refusals(kw, status):
    c = cache(**kw)
    r = rows(sb=2 * 64, sh=64)
    p = ctypes.c_void_p(GOOD)
    L = lh.LIB
    H = max(c.H, 1)
    k = lh.LhRows(GOOD, 4096, 64, 64, H)
    assert L.lh_cache_append(ctypes.byref(c), None, 1, ctypes.byref(k), ctypes.byref(k), None, None, None, 0,
                             None, None, None) == status
    assert L.lh_decode(ctypes.byref(c), ctypes.byref(r), 0.125, p, p, None, None, p, 1 << 30, None) == status
    assert L.lh_evict(ctypes.byref(c), 4, p, None, None, p, None, ctypes.c_void_p(GOOD << 2), p, 1 << 40,
                      None) == status


def test_append_refusals():
    c, bad = cache(), lh.LH_ERR_INVALID_ARG

    def call(K=None, V=None, Q=None, Qo=None, T=8, rotary=None, counts=None, positions=None, slot=None):
        ref = [None if r is None else ctypes.byref(r) for r in
               (rows() if K is None else K, rows() if V is None else V, Q, Qo)]
        return lh.LIB.lh_cache_append(ctypes.byref(c), None if rotary is None else ctypes.byref(rotary), T, *ref,
                                      positions, 0, counts, slot, None)

    assert call(T=-1) == bad and call(T=1 << 31) == bad
    assert call(K=rows(H=4, sb=4 * 512)) == bad and call(V=rows(H=1)) == bad
    assert call(Q=rows()) == bad and call(Qo=rows()) == bad
    assert call(Q=rows(), Qo=rows(ptr=GOOD + 128)) == bad
    for q, out in ((GOOD << 4, GOOD), (GOOD << 4, c.v)):           # queries into the new keys, into the cache
        assert call(Q=rows(ptr=q), Qo=rows(ptr=out)) == bad and b"Qo" in lh.LIB.lh_last_error()
    assert call(K=rows(sh=12)) == bad
    assert call(rotary=lh.rotary_plan(128).raw) == bad
    for name in ("counts", "positions", "slot"):
        assert call(**{name: ctypes.c_void_p(GOOD + 1)}) == bad
    assert call(T=0) == lh.LH_OK


def test_decode_refusals():
    c, bad = cache(), lh.LH_ERR_INVALID_ARG
    p = ctypes.c_void_p(GOOD)
    need = lh.LIB.lh_decode_ws_bytes(ctypes.byref(c), 4, 1)
    assert need > lh.LIB.lh_decode_ws_bytes(ctypes.byref(c), 4, 0) > 0
    assert lh.LIB.lh_decode_ws_bytes(ctypes.byref(c), 3, 0) == -1
    assert lh.LIB.lh_decode_ws_bytes(ctypes.byref(cache(page=17)), 4, 0) == -1

    def call(q=None, scale=0.125, o=p, lse=p, w=None, wo=None, ws=p, n=need):
        q = rows(H=4, sb=4 * 64, sh=64) if q is None else q
        return lh.LIB.lh_decode(ctypes.byref(c), ctypes.byref(q), scale, o, lse, w, wo, ws, n, None)

    assert call(q=rows(H=3)) == bad and call(q=rows(H=4, sh=20)) == bad
    assert call(scale=float("inf")) == bad and call(scale=3e38) == bad and call(scale=float("nan")) == bad
    assert call(o=None) == bad and call(lse=None) == bad
    assert call(w=p) == bad and call(wo=p) == bad
    assert call(w=p, wo=ctypes.c_void_p(GOOD + 64)) == bad      # shifted: overlaps
    assert call(ws=None) == bad
    assert call(w=p, wo=p, n=need - 1) == lh.LH_ERR_WORKSPACE
    assert call(n=0) == lh.LH_ERR_WORKSPACE


def test_evict_refusals():
    c, bad = cache(), lh.LH_ERR_INVALID_ARG
    p, apart = ctypes.c_void_p(GOOD), ctypes.c_void_p(GOOD << 1)
    need = lh.LIB.lh_evict_ws_bytes(ctypes.byref(c), 16)
    assert need > 0 and lh.LIB.lh_evict_ws_bytes(ctypes.byref(c), 0) == -1

    def call(budget=16, w=p, pos=None, prot=None, wo=p, po=None, n=apart, ws=p, size=need):
        return lh.LIB.lh_evict(ctypes.byref(c), budget, w, pos, prot, wo, po, n, ws, size, None)

    assert call(budget=0) == bad and call(budget=-5) == bad
    assert call(w=None) == bad and call(wo=None) == bad and call(n=None) == bad
    assert call(pos=p) == bad and call(po=p) == bad
    assert call(n=p) == bad and b"lengths" in lh.LIB.lh_last_error()   # the cache's own lengths
    assert call(wo=ctypes.c_void_p(GOOD + 16)) == bad
    assert call(pos=p, po=ctypes.c_void_p(GOOD + 16)) == bad
    assert call(prot=ctypes.c_void_p(GOOD + 1)) == bad
    assert call(size=need - 1) == lh.LH_ERR_WORKSPACE


def test_binding_checks_cache_arguments_before_calling_the_library():
    bf, i32 = torch.bfloat16, torch.int32
    rp = lh.rotary_plan(64)
    x = torch.zeros(2, 4, 8, 64, dtype=bf)
    kc = lh.PagedCache.of(torch.zeros(8, 2, 16, 64, dtype=bf), torch.zeros(8, 2, 16, 64, dtype=bf))
    table, lens = torch.zeros(2, 4, dtype=i32), torch.zeros(2, dtype=i32)
    new = torch.zeros(2, 2, 3, 64, dtype=bf)
    q = torch.zeros(2, 4, 1, 64, dtype=bf)
    w = torch.zeros(2, 2, 64)
    p = torch.zeros(2, 2, 64, dtype=i32)
    cases = [
        (lambda: lh.rotary(rp, x.half()), "dtype"),
        (lambda: lh.rotary(rp, x[0]), "[B, H, N, d]"),
        (lambda: lh.rotary(rp, x, x.float()), "dtype"),
        (lambda: lh.rotary(rp, x, x[:, :, :7]), "shape"),
        (lambda: lh.rotary(lh.rotary_plan(128), x), "shape"),
        (lambda: lh.rotary(rp, x.transpose(2, 3).contiguous().transpose(2, 3)), "channels"),
        (lambda: lh.rotary(rp, x, positions=torch.zeros(8, dtype=torch.int64)), "dtype"),
        (lambda: lh.rotary(rp, x, positions=torch.zeros(3, 8, dtype=i32)), "shape"),
        (lambda: lh.rotary(rp, x, x, out=(x,)), "two tensors"),
        (lambda: lh.rotary(rp, x, out=x[:, :2]), "shape"),
        (lambda: lh.rotary(rp, x), "CUDA"),
        (lambda: lh.rotary_bwd(rp, x, x), "CUDA"),
        (lambda: lh.PagedCache.of(x.half(), x.half()), "dtype"),
        (lambda: lh.PagedCache.of(x, x[:, :2]), "shape"),
        (lambda: lh.PagedCache.of(x.transpose(1, 2), x.transpose(1, 2)), "contiguous"),
        (lambda: lh.cache_append(kc, table.long(), lens, new, new), "table: dtype"),
        (lambda: lh.cache_append(kc, table[0], lens, new, new), "[B, width]"),
        (lambda: lh.cache_append(kc, table, lens[:1], new, new), "lengths: shape"),
        (lambda: lh.cache_append(kc, table, lens, new[:, :1], new), "K: shape"),
        (lambda: lh.cache_append(kc, table, lens, new, new.float()), "V: dtype"),
        (lambda: lh.cache_append(kc, table, lens, new, new, out=q), "without Q"),
        (lambda: lh.cache_append(kc, table, lens, new, new, Q=q), "Q: shape"),
        (lambda: lh.cache_append(kc, table, lens, new, new, counts=lens.long()), "counts: dtype"),
        (lambda: lh.cache_append(kc, table, lens, new, new, slot_positions=p[:1]), "slot_positions: shape"),
        (lambda: lh.cache_append(kc, table, lens, new, new, rotary=lh.rotary_plan(128)), "rotary"),
        (lambda: lh.cache_append(kc, table, lens, new, new), "CUDA"),
        (lambda: lh.decode(kc, table, lens, q[:, :, 0]), "Q: shape"),
        (lambda: lh.decode(kc, table, lens, q.float()), "Q: dtype"),
        (lambda: lh.decode(kc, table, lens, q, weights_out=w), "without weights"),
        (lambda: lh.decode(kc, table, lens, q, weights=w[:, :, :63]), "weights: shape"),
        (lambda: lh.decode(kc, table, lens, q, weights=w.double()), "weights: dtype"),
        (lambda: lh.decode(kc, table, lens, q, ws=torch.zeros(4, dtype=torch.uint8)), "elements"),
        (lambda: lh.decode(kc, table, lens, q), "CUDA"),
        (lambda: lh.evict(kc, table, lens, w[:1], 8), "weights: shape"),
        (lambda: lh.evict(kc, table, lens, w, 8, positions=p.long()), "positions: dtype"),
        (lambda: lh.evict(kc, table, lens, w, 8, positions_out=p), "without positions"),
        (lambda: lh.evict(kc, table, lens, w, 8, protect=lens.float()), "protect: dtype"),
        (lambda: lh.evict(kc, table, lens, w, 8), "CUDA"),
    ]
    for call, what in cases:
        with pytest.raises((ValueError, TypeError)) as e:
            call()
        assert what in str(e.value), (what, str(e.value))
    with pytest.raises(lh.LighthouseError):
        lh.decode(kc, table, lens, torch.zeros(2, 3, 1, 64, dtype=bf))  # 3 query heads on 2 key heads
    with pytest.raises(lh.LighthouseError):
        lh.evict(kc, table, lens, w, 0)


def test_workspace_sizes_follow_the_shapes():
    table, lens = torch.zeros(2, 4, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    kc = lh.PagedCache.of(*(torch.zeros(8, 2, 16, 64, dtype=torch.bfloat16) for _ in range(2)))
    plain, more = (lh.decode_ws_bytes(kc, table, lens, 4, w) for w in (False, True))
    assert more == plain + 2 * 4 * 64 * 4
    assert lh.evict_ws_bytes(kc, table, lens, 64) < lh.evict_ws_bytes(kc, table, lens, 32)


def test_size_queries_refuse_with_the_status_of_their_calls():
    """What a call refuses as not built is not reported as an invalid argument by the scratch
    size that the binding asks for before it, and the other way round."""
    i32, bf = torch.int32, torch.bfloat16
    table, lens = torch.zeros(2, 4, dtype=i32), torch.zeros(2, dtype=i32)

    def kc(H=2, page=16, d=64):
        return lh.PagedCache.of(*(torch.zeros(8, H, page, d, dtype=bf) for _ in range(2)))

    for cache_, status in ((kc(page=48), lh.LH_ERR_UNSUPPORTED), (kc(d=32), lh.LH_ERR_UNSUPPORTED),
                           (kc(H=0), lh.LH_ERR_INVALID_ARG)):
        H, page, d = cache_.H, cache_.page, cache_.d
        w = torch.zeros(2, H, 4 * page)
        for call in (lambda: lh.decode(cache_, table, lens, torch.zeros(2, 2, 1, d, dtype=bf)),
                     lambda: lh.decode_ws_bytes(cache_, table, lens, 2),
                     lambda: lh.evict(cache_, table, lens, w, 8), lambda: lh.evict_ws_bytes(cache_, table, lens, 8)):
            with pytest.raises(lh.LighthouseError) as e:
                call()
            assert e.value.status == status, str(e.value)
    for call, status in ((lambda: lh.decode_ws_bytes(kc(), table, lens, 3), lh.LH_ERR_INVALID_ARG),
                         (lambda: lh.decode_ws_bytes(kc(), table, lens, 1 << 22), lh.LH_ERR_UNSUPPORTED),
                         (lambda: lh.evict_ws_bytes(kc(), table, lens, 0), lh.LH_ERR_INVALID_ARG)):
        with pytest.raises(lh.LighthouseError) as e:
            call()
        assert e.value.status == status, str(e.value)
    assert lh.LIB.lh_decode_ws_bytes(ctypes.byref(cache(page=17)), 4, 0) == -1
    assert lh.LIB.lh_last_status() == lh.LH_ERR_UNSUPPORTED
    assert lh.LIB.lh_evict_ws_bytes(ctypes.byref(cache()), 0) == -1
    assert lh.LIB.lh_last_status() == lh.LH_ERR_INVALID_ARG


def test_positions_without_rotary_are_refused():
    """The layer would leave them unused, and its caller expects rows to be turned."""
    pl = lh.plan(1, 2, 64, 64, 4, 2, 2, "bf16")
    x = torch.zeros(1, 2, 64, 64, dtype=torch.bfloat16)
    for kw in (dict(positions=torch.zeros(64, dtype=torch.int32)), dict(start=5)):
        with pytest.raises(ValueError) as e:
            lh.forward(pl, x, x, x, **kw)
        assert "rotary" in str(e.value)
    with pytest.raises(ValueError) as e:
        lh.forward(pl, x, x, x)
    assert "CUDA" in str(e.value)
