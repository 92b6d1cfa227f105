"""Python binding of the Lighthouse C ABI (include/lh.h).

Argument marshalling only: every stage runs in liblh.so's CUDA kernels.
PyTorch provides device memory and the current stream.  Importing this module
loads liblh.so and fails loudly if it is missing; there is no fallback.
"""
from __future__ import annotations

import ctypes
import os
import struct
from dataclasses import dataclass

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
# LH_LIBRARY selects another build of the library (for example a variant
# compiled with different tile constants); the default is the in-tree one.
LIB_PATH = os.environ.get("LH_LIBRARY") or os.path.join(HERE, "liblh.so")

(LH_OK, LH_ERR_INVALID_ARG, LH_ERR_UNSUPPORTED, LH_ERR_WORKSPACE, LH_ERR_CUDA, LH_ERR_TIMEOUT,
 LH_ERR_PAGE) = range(7)
LH_F32, LH_BF16 = 0, 1
MAX_LEVELS = 8
DTYPES = {"f32": LH_F32, "bf16": LH_BF16}
TORCH_DTYPE = {LH_F32: torch.float32, LH_BF16: torch.bfloat16}

# Every exported name declared in include/lh.h.
EXPORTS = (
    "lh_plan_init", "lh_pyramid", "lh_score", "lh_pyramid_score", "lh_topk", "lh_gather",
    "lh_attn_fwd", "lh_attn_bwd_ws_bytes", "lh_attn_bwd", "lh_scatter", "lh_scatter_bwd",
    "lh_gather_bwd", "lh_forward", "lh_backward", "lh_device_status", "lh_status_string",
    "lh_last_error", "lh_plan_bytes", "lh_attn_bwd_static", "lh_set_deterministic",
    "lh_selftest_wait_timeout", "lh_rotary_init", "lh_rotary_plan_bytes", "lh_rotary",
    "lh_cache_bytes", "lh_cache_append", "lh_decode_ws_bytes", "lh_decode", "lh_evict_ws_bytes",
    "lh_evict", "lh_last_status",
)


SELECT = {"joint": 0, "descent": 1, "regional": 2}


class LhConfig(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("B", "H", "N", "d", "p", "L", "k", "dtype", "select")]


_I64 = ctypes.c_int64


class LhPlan(ctypes.Structure):
    _fields_ = [
        ("c", LhConfig),
        ("P", _I64 * MAX_LEVELS),
        ("n", _I64 * MAX_LEVELS),
        ("flat_off", _I64 * (MAX_LEVELS + 1)),
        ("pyr_off", _I64 * MAX_LEVELS),
    ] + [(n, _I64) for n in (
        "Ntot", "Npyr", "M", "Ksel", "S", "elem_bytes",
        "ctx_bytes", "ws_bytes", "topk_ws_bytes", "attn_bwd_ws_bytes",
        "ctx_sel_idx", "ctx_slot_of", "ctx_Qg", "ctx_Kg", "ctx_Vg", "ctx_Og", "ctx_lse",
        "ws_pyrQ", "ws_pyrK", "ws_pyrV", "ws_scores", "ws_topk",
        "ws_dOg", "ws_D", "ws_dQg", "ws_dKg", "ws_dVg", "ws_attn")]


MAX_PAIRS = 64
LAYOUT = {"half": 0, "interleaved": 1}
SCALING = {"none": 0, "linear": 1, "bands": 2}
_I32, _F64 = ctypes.c_int32, ctypes.c_double


class LhRotaryConfig(ctypes.Structure):
    _fields_ = [(n, _I32) for n in ("d", "rot", "layout", "scaling")] + \
        [(n, _F64) for n in ("base", "factor", "low", "high", "original", "magnitude")]


class LhRotaryPlan(ctypes.Structure):
    _fields_ = [("c", LhRotaryConfig), ("turns", ctypes.c_uint64 * MAX_PAIRS),
                ("check", ctypes.c_uint64)]


class LhRows(ctypes.Structure):
    _fields_ = [("ptr", ctypes.c_void_p), ("stride_b", _I64), ("stride_h", _I64), ("stride_n", _I64),
                ("H", _I64)]


class LhCache(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("pages", _I64), ("H", _I32),
                ("page", _I32), ("d", _I32), ("dtype", _I32), ("table", ctypes.c_void_p),
                ("table_stride", _I64), ("B", _I32), ("width", _I32), ("lengths", ctypes.c_void_p)]


class LighthouseError(RuntimeError):
    def __init__(self, status: int, where: str, detail: str):
        self.status = status
        super().__init__(f"{where}: status {status} ({detail})")


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(
            f"{LIB_PATH} is missing: build it with `python -m long_context_hierarchical_b200.build`"
            " (the Lighthouse layer has no CPU fallback)")
    lib = ctypes.CDLL(LIB_PATH)
    P, I64, I32, SZ = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_size_t
    PLAN = ctypes.POINTER(LhPlan)
    sig = {
        "lh_plan_init": (ctypes.POINTER(LhConfig), PLAN),
        "lh_pyramid": (PLAN, P, P, P, P, P, P, P),
        "lh_score": (PLAN, P, P, P, P),
        "lh_pyramid_score": (PLAN, P, P, P, P, P, P, P, P),
        "lh_topk": (PLAN, P, P, P, P, SZ, P),
        "lh_gather": (PLAN, P, P, P, P, P, P, P, P, P, P, P),
        "lh_attn_fwd": (I64, I64, I32, I32, P, P, P, P, P, P),
        "lh_attn_bwd": (I64, I64, I32, I32, P, P, P, P, P, P, P, P, P, P, P, SZ, P),
        "lh_scatter": (PLAN, P, P, P, P),
        "lh_scatter_bwd": (PLAN, P, P, P, P, P, P),
        "lh_gather_bwd": (PLAN, P, P, P, P, P, P, P, P),
        "lh_forward": (PLAN, P, P, P, P, P, SZ, P, SZ, P),
        "lh_backward": (PLAN, P, P, SZ, P, P, P, P, SZ, P),
        "lh_device_status": (ctypes.c_int,),
        "lh_selftest_wait_timeout": (P,),
        "lh_attn_bwd_static": (I64, I64, I32, I32, P, P, P, P, P, P, P, P, P, P),
        "lh_rotary_init": (ctypes.POINTER(LhRotaryConfig), ctypes.POINTER(LhRotaryPlan)),
        "lh_rotary": (ctypes.POINTER(LhRotaryPlan), I32, I64, I64, I32, P, P, P, I64, I64, I32, P),
        "lh_cache_append": (P, P, I64, P, P, P, P, P, I64, P, P, P),
        "lh_decode": (P, P, ctypes.c_float, P, P, P, P, P, SZ, P),
        "lh_evict": (P, I64, P, P, P, P, P, P, P, SZ, P),
    }
    for name, args in sig.items():
        f = getattr(lib, name)
        f.argtypes = list(args)
        f.restype = ctypes.c_int
    lib.lh_attn_bwd_ws_bytes.argtypes = [I64, I64, I32, I32]
    lib.lh_attn_bwd_ws_bytes.restype = I64
    lib.lh_status_string.argtypes = [ctypes.c_int]
    lib.lh_status_string.restype = ctypes.c_char_p
    lib.lh_last_error.argtypes = []
    lib.lh_last_error.restype = ctypes.c_char_p
    lib.lh_last_status.argtypes = []
    lib.lh_last_status.restype = ctypes.c_int
    lib.lh_plan_bytes.argtypes = []
    lib.lh_plan_bytes.restype = I64
    lib.lh_set_deterministic.argtypes = [ctypes.c_int]
    lib.lh_set_deterministic.restype = None
    lib.lh_decode_ws_bytes.argtypes = [P, I64, I32]
    lib.lh_evict_ws_bytes.argtypes = [P, I64]
    for name in ("lh_decode_ws_bytes", "lh_evict_ws_bytes", "lh_rotary_plan_bytes", "lh_cache_bytes"):
        getattr(lib, name).restype = I64
    if lib.lh_plan_bytes() != ctypes.sizeof(LhPlan):
        raise ImportError("lh_plan layout of liblh.so does not match this binding")
    if lib.lh_rotary_plan_bytes() != ctypes.sizeof(LhRotaryPlan) or \
            lib.lh_cache_bytes() != ctypes.sizeof(LhCache):
        raise ImportError("lh_rotary_plan or lh_cache layout of liblh.so does not match this binding")
    return lib


LIB = _load()


def _check(status: int, where: str):
    if status != LH_OK:
        detail = (LIB.lh_last_error() or b"").decode() or LIB.lh_status_string(status).decode()
        raise LighthouseError(status, where, detail)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _require(t, name: str, dtype, numel: int):
    """Check a tensor the library will read or write as ``numel`` contiguous
    elements of ``dtype`` in device memory (the C ABI sees only its pointer)."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor, got {type(t).__name__}")
    if t.dtype != dtype:
        raise ValueError(f"{name}: dtype {t.dtype}, expected {dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")
    if t.numel() < numel:
        raise ValueError(f"{name}: {t.numel()} elements, the call needs {numel}")
    if t.device.type != "cuda":
        raise ValueError(f"{name}: must be a CUDA tensor (got {t.device})")


def _require_tokens(pl, **tensors):
    """[B,H,N,d] tensors of the plan's dtype."""
    c = pl.raw.c
    for name, t in tensors.items():
        _require(t, name, pl.dtype, c.B * c.H * c.N * c.d)


def _require_rows(pl, **tensors):
    """[B,H,S,d] gathered tensors of the plan's dtype."""
    c = pl.raw.c
    for name, t in tensors.items():
        _require(t, name, pl.dtype, c.B * c.H * pl.S * c.d)


def _attn_shape(Qg, **others):
    """(BH, S, d) of [..., S, d] attention operands; every other operand has
    Qg's dtype and size."""
    if not isinstance(Qg, torch.Tensor) or Qg.dim() < 2:
        raise ValueError("Qg: expected a tensor of shape [..., S, d]")
    if Qg.dtype not in (torch.bfloat16, torch.float32):
        raise ValueError(f"Qg: dtype {Qg.dtype}, expected torch.bfloat16 or torch.float32")
    S, d = Qg.shape[-2], Qg.shape[-1]
    _require(Qg, "Qg", Qg.dtype, Qg.numel())
    for name, t in others.items():
        _require(t, name, Qg.dtype, Qg.numel())
    return Qg.numel() // max(S * d, 1), S, d


def _stream(stream=None):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


@dataclass
class Plan:
    """Sizes and buffer layout of one layer configuration (from lh_plan_init)."""
    raw: LhPlan

    @property
    def S(self):
        return self.raw.S

    @property
    def M(self):
        return self.raw.M

    @property
    def Ntot(self):
        return self.raw.Ntot

    @property
    def Npyr(self):
        return self.raw.Npyr

    @property
    def Ksel(self):
        return self.raw.Ksel

    @property
    def BH(self):
        return self.raw.c.B * self.raw.c.H

    @property
    def dtype(self):
        return TORCH_DTYPE[self.raw.c.dtype]

    def byref(self):
        return ctypes.byref(self.raw)


def plan(B: int, H: int, N: int, d: int = 64, p: int = 4, L: int = 3, k: int = 0,
         dtype: str = "bf16", select: str = "joint") -> Plan:
    """select: "joint" (one top-K over all candidate levels), "descent"
    (hierarchical descent from the coarsest level) or "regional" (every
    2048-candidate region keeps its share of the budget)."""
    cfg = LhConfig(B, H, N, d, p, L, k, DTYPES[dtype], SELECT[select])
    raw = LhPlan()
    _check(LIB.lh_plan_init(ctypes.byref(cfg), ctypes.byref(raw)), "lh_plan_init")
    return Plan(raw)


def _empty(shape, dtype, device):
    return torch.empty(shape, dtype=dtype, device=device)


def _bytes(n, device):
    return torch.empty(max(int(n), 16), dtype=torch.uint8, device=device)


# --- stages -----------------------------------------------------------------


def pyramid_score(pl: Plan, Q, K, V, stream=None):
    """Levels 1..L-1 of Q, K, V ([B,H,Npyr,d] each) and candidate scores [B,H,M]."""
    _require_tokens(pl, Q=Q, K=K, V=V)
    c = pl.raw.c
    dev = Q.device
    pyr = [_empty((c.B, c.H, max(pl.Npyr, 1), c.d), Q.dtype, dev) for _ in range(3)]
    scores = _empty((c.B, c.H, max(pl.M, 1)), torch.float32, dev)
    _check(LIB.lh_pyramid_score(pl.byref(), _ptr(Q), _ptr(K), _ptr(V), *map(_ptr, pyr),
                                _ptr(scores), _stream(stream)), "lh_pyramid_score")
    return pyr, scores


def pyramid(pl: Plan, Q, K, V, stream=None):
    _require_tokens(pl, Q=Q, K=K, V=V)
    c = pl.raw.c
    pyr = [_empty((c.B, c.H, max(pl.Npyr, 1), c.d), Q.dtype, Q.device) for _ in range(3)]
    _check(LIB.lh_pyramid(pl.byref(), _ptr(Q), _ptr(K), _ptr(V), *map(_ptr, pyr),
                          _stream(stream)), "lh_pyramid")
    return pyr


def score(pl: Plan, Q, K, stream=None):
    _require_tokens(pl, Q=Q, K=K)
    c = pl.raw.c
    scores = _empty((c.B, c.H, max(pl.M, 1)), torch.float32, Q.device)
    _check(LIB.lh_score(pl.byref(), _ptr(Q), _ptr(K), _ptr(scores), _stream(stream)), "lh_score")
    return scores


def topk(pl: Plan, scores, stream=None):
    """(sel_idx [B,H,S] int32, slot_of [B,H,Ntot] int32) from scores [B,H,M]."""
    c = pl.raw.c
    _require(scores, "scores", torch.float32, c.B * c.H * pl.M)
    dev = scores.device
    sel = _empty((c.B, c.H, pl.S), torch.int32, dev)
    inv = _empty((c.B, c.H, pl.Ntot), torch.int32, dev)
    ws = _bytes(pl.raw.topk_ws_bytes, dev)
    _check(LIB.lh_topk(pl.byref(), _ptr(scores), _ptr(sel), _ptr(inv), _ptr(ws), ws.numel(),
                       _stream(stream)), "lh_topk")
    return sel, inv


def gather(pl: Plan, Q, K, V, pyr, sel_idx, stream=None):
    _require_tokens(pl, Q=Q, K=K, V=V)
    c = pl.raw.c
    if len(pyr) != 3:
        raise ValueError("pyr: expected the three pyramids (Q, K, V)")
    for name, t in zip(("pyrQ", "pyrK", "pyrV"), pyr):
        _require(t, name, pl.dtype, c.B * c.H * pl.Npyr * c.d)
    _require(sel_idx, "sel_idx", torch.int32, c.B * c.H * pl.S)
    out = [_empty((c.B, c.H, pl.S, c.d), Q.dtype, Q.device) for _ in range(3)]
    _check(LIB.lh_gather(pl.byref(), _ptr(Q), _ptr(K), _ptr(V), *map(_ptr, pyr), _ptr(sel_idx),
                         *map(_ptr, out), _stream(stream)), "lh_gather")
    return out


def _dtype_code(t):
    return LH_BF16 if t.dtype == torch.bfloat16 else LH_F32


def attn_fwd(Qg, Kg, Vg, stream=None):
    """Causal attention on [..., S, d] tensors: (O, lse[..., S] natural log)."""
    BH, S, d = _attn_shape(Qg, Kg=Kg, Vg=Vg)
    O = torch.empty_like(Qg)
    lse = _empty(Qg.shape[:-1], torch.float32, Qg.device)
    _check(LIB.lh_attn_fwd(BH, S, d, _dtype_code(Qg), _ptr(Qg), _ptr(Kg), _ptr(Vg), _ptr(O),
                           _ptr(lse), _stream(stream)), "lh_attn_fwd")
    return O, lse


def attn_bwd(Qg, Kg, Vg, Og, lse, dOg, D=None, stream=None):
    BH, S, d = _attn_shape(Qg, Kg=Kg, Vg=Vg, Og=Og, dOg=dOg)
    _require(lse, "lse", torch.float32, BH * S)
    if D is not None:
        _require(D, "D", torch.float32, BH * S)
    code = _dtype_code(Qg)
    dQ, dK, dV = torch.empty_like(Qg), torch.empty_like(Kg), torch.empty_like(Vg)
    ws = _bytes(LIB.lh_attn_bwd_ws_bytes(BH, S, d, code), Qg.device)
    _check(LIB.lh_attn_bwd(BH, S, d, code, _ptr(Qg), _ptr(Kg), _ptr(Vg), _ptr(Og), _ptr(lse),
                           _ptr(dOg), _ptr(D), _ptr(dQ), _ptr(dK), _ptr(dV), _ptr(ws), ws.numel(),
                           _stream(stream)), "lh_attn_bwd")
    return dQ, dK, dV


def attn_bwd_static(Qg, Kg, Vg, Og, lse, dOg, stream=None):
    """lh_attn_bwd with D computed into the library's own scratch array
    (no workspace: for callers that cannot allocate device memory)."""
    BH, S, d = _attn_shape(Qg, Kg=Kg, Vg=Vg, Og=Og, dOg=dOg)
    _require(lse, "lse", torch.float32, BH * S)
    dQ, dK, dV = torch.empty_like(Qg), torch.empty_like(Kg), torch.empty_like(Vg)
    _check(LIB.lh_attn_bwd_static(BH, S, d, _dtype_code(Qg), _ptr(Qg), _ptr(Kg), _ptr(Vg), _ptr(Og),
                                  _ptr(lse), _ptr(dOg), _ptr(dQ), _ptr(dK), _ptr(dV),
                                  _stream(stream)), "lh_attn_bwd_static")
    return dQ, dK, dV


def scatter(pl: Plan, Og, slot_of, stream=None):
    _require_rows(pl, Og=Og)
    c = pl.raw.c
    _require(slot_of, "slot_of", torch.int32, c.B * c.H * pl.Ntot)
    O = _empty((c.B, c.H, c.N, c.d), Og.dtype, Og.device)
    _check(LIB.lh_scatter(pl.byref(), _ptr(Og), _ptr(slot_of), _ptr(O), _stream(stream)),
           "lh_scatter")
    return O


def scatter_bwd(pl: Plan, dO, Og, sel_idx, stream=None):
    _require_tokens(pl, dO=dO)
    _require_rows(pl, Og=Og)
    c = pl.raw.c
    _require(sel_idx, "sel_idx", torch.int32, c.B * c.H * pl.S)
    dOg = _empty((c.B, c.H, pl.S, c.d), dO.dtype, dO.device)
    D = _empty((c.B, c.H, pl.S), torch.float32, dO.device)
    _check(LIB.lh_scatter_bwd(pl.byref(), _ptr(dO), _ptr(Og), _ptr(sel_idx), _ptr(dOg), _ptr(D),
                              _stream(stream)), "lh_scatter_bwd")
    return dOg, D


def gather_bwd(pl: Plan, dQg, dKg, dVg, slot_of, stream=None):
    _require_rows(pl, dQg=dQg, dKg=dKg, dVg=dVg)
    c = pl.raw.c
    _require(slot_of, "slot_of", torch.int32, c.B * c.H * pl.Ntot)
    out = [_empty((c.B, c.H, c.N, c.d), dQg.dtype, dQg.device) for _ in range(3)]
    _check(LIB.lh_gather_bwd(pl.byref(), _ptr(dQg), _ptr(dKg), _ptr(dVg), _ptr(slot_of),
                             *map(_ptr, out), _stream(stream)), "lh_gather_bwd")
    return out


# --- rotary positions ---------------------------------------------------------


# The device's current stream as an integer handle (a Stream object costs more
# to make than a small call takes on the GPU).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda index: torch.cuda.current_stream(index).cuda_stream)


def _run(dev, stream, inputs, call):
    """``call(handle)`` enqueues on ``stream`` (default: the device's current one)
    and returns the tensors it allocated, with ``dev`` as the current device.

    On a stream other than the current one the outputs come from that stream's
    memory pool, and every tensor is recorded on the stream it is used on next
    to its own, so that none is handed out again while the other one works."""
    if stream is None:
        if dev.index == torch.cuda.current_device():
            return call(_raw_stream(dev.index))
        with torch.cuda.device(dev):
            return call(_raw_stream(dev.index))
    cur = torch.cuda.current_stream(dev)
    if stream == cur:
        return _run(dev, None, inputs, call)
    if stream.device != dev:
        raise ValueError(f"stream: on {stream.device}, the tensors are on {dev}")
    with torch.cuda.stream(stream):
        outs = call(stream.cuda_stream)
    for t in inputs:
        if t is not None:
            t.record_stream(stream)
    for t in outs:
        if t is not None:
            t.record_stream(cur)
    return outs


def _on_device(dev, names, tensors):
    """All tensors of the call (those that are not None) are on the CUDA device ``dev``."""
    if dev.type != "cuda":
        raise ValueError(f"{names.split()[0]}: must be a CUDA tensor (got {dev})")
    index = dev.index
    for i, t in enumerate(tensors):
        if t is not None and t.get_device() != index:
            raise ValueError(f"{names.split()[i]}: on {t.device}, the call runs on {dev}")


def _rows_of(t, name: str, dtype, B, H, N, d):
    """Check a [B, H, N, d] tensor (any H where H is None) that the library reads
    or writes by its strides; returns the five fields of its lh_rows."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor, got {type(t).__name__}")
    if t.dtype != dtype:
        raise ValueError(f"{name}: dtype {t.dtype}, expected {dtype}")
    have = t.shape
    if have != (B, have[1] if H is None and len(have) == 4 else H, N, d):
        want = ", ".join("*" if w is None else str(w) for w in (B, H, N, d))
        raise ValueError(f"{name}: shape {tuple(have)}, expected [{want}]")
    sb, sh, sn, sc = t.stride()
    if sc != 1:
        raise ValueError(f"{name}: the channels of a row must be contiguous")
    return t.data_ptr(), sb, sh, sn, have[1]


# An lh_rows, one or two side by side, and the two halves of an lh_cache, packed: a
# ctypes object made for every call takes several times as long.
_ROW = struct.Struct("P4q").pack
_ROWS = (None, _ROW, struct.Struct("P4qP4q").pack)
_PAGES = struct.Struct("PPq4i").pack    # k, v, pages, H, page, d, dtype
_BATCH = struct.Struct("PqiiP").pack    # table, table_stride, B, width, lengths


def _index(t, name: str, shape):
    """Check an int32 index tensor."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor, got {type(t).__name__}")
    if t.dtype != torch.int32:
        raise ValueError(f"{name}: dtype {t.dtype}, expected torch.int32")
    if t.shape != shape:
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {list(shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")


def _positions(t, B: int, N: int):
    """Row stride of a positions tensor of shape [N], [1, N] or [B, N]."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"positions: expected a torch.Tensor, got {type(t).__name__}")
    if t.dtype != torch.int32:
        raise ValueError(f"positions: dtype {t.dtype}, expected torch.int32")
    if tuple(t.shape) not in ((N,), (1, N), (B, N)):
        raise ValueError(f"positions: shape {tuple(t.shape)}, expected [{N}] or [{B}, {N}]")
    if N > 1 and t.stride(-1) != 1:
        raise ValueError("positions: a sequence's positions must be contiguous")
    return t.stride(0) if t.dim() == 2 and t.shape[0] > 1 else 0


@dataclass
class RotaryPlan:
    """Frequencies and pair layout of a rotation (from lh_rotary_init)."""
    raw: LhRotaryPlan

    def __post_init__(self):
        self.d = self.raw.c.d


def rotary_plan(d: int = 64, rot: int | None = None, base: float = 10000.0, layout: str = "half",
                scaling: str = "none", factor: float = 1.0, low: float = 1.0, high: float = 4.0,
                original: float = 0.0, magnitude: float = 1.0) -> RotaryPlan:
    """rot: turned channels (default all d); layout: "half" pairs channels
    (i, i + rot/2), "interleaved" (2i, 2i + 1); scaling: "none", "linear"
    (every frequency divided by factor) or "bands" (slow pairs divided, fast
    ones kept: those that make more than ``high`` turns in ``original``
    positions, with a ramp down to ``low``); magnitude multiplies every turned channel."""
    cfg = LhRotaryConfig(d, d if rot is None else rot, LAYOUT[layout], SCALING[scaling], base, factor,
                         low, high, original, magnitude)
    raw = LhRotaryPlan()
    _check(LIB.lh_rotary_init(ctypes.byref(cfg), ctypes.byref(raw)), "lh_rotary_init")
    return RotaryPlan(raw)


def _dense_rows(t):
    """The lh_rows fields of a contiguous [B, H, N, d] tensor."""
    _, H, N, d = t.shape
    return t.data_ptr(), H * N * d, N * d, d, H


def _contiguous_like(t):
    return torch.empty_like(t) if t.is_contiguous() else \
        torch.empty_like(t, memory_format=torch.contiguous_format)


def _rotate(rp: RotaryPlan, X, Y, positions, start, transpose, stream):
    """Turn the one or two tensors X into Y (None: new contiguous tensors)."""
    first = X[0]
    if not isinstance(first, torch.Tensor) or first.dim() != 4:
        raise ValueError("Q: expected a tensor of shape [B, H, N, d]")
    if first.dtype not in (torch.bfloat16, torch.float32):
        raise ValueError(f"Q: dtype {first.dtype}, expected torch.bfloat16 or torch.float32")
    B, _, N, _ = first.shape
    d = rp.d
    x = ()
    y = ()
    for i, t in enumerate(X):
        x += _rows_of(t, "QK"[i], first.dtype, B, None, N, d)
        if Y is not None:
            y += _rows_of(Y[i], f"out[{i}]", first.dtype, B, t.shape[1], N, d)
    stride = 0 if positions is None else _positions(positions, B, N)
    dev = first.device
    tensors = (*X, positions) if Y is None else (*X, positions, *Y)
    _on_device(dev, "Q positions out" if len(X) == 1 else "Q K positions out[0] out[1]", tensors)

    def call(handle):
        out, rows = Y, y
        if Y is None:
            out = tuple([_contiguous_like(t) for t in X])
            for t in out:
                rows += _dense_rows(t)
        if B and N:
            n = len(X)
            _check(LIB.lh_rotary(ctypes.byref(rp.raw), _dtype_code(first), B, N, n, _ROWS[n](*x), _ROWS[n](*rows),
                                 _ptr(positions), stride, start, transpose, handle), "lh_rotary")
        return out

    return _run(dev, stream, tensors, call)


def _pair(Q, K, out):
    if K is None:
        return (Q,), None if out is None else (out,)
    if out is not None and len(out) != 2:
        raise ValueError("out: expected two tensors")
    return (Q, K), None if out is None else tuple(out)


def rotary(rp: RotaryPlan, Q, K=None, positions=None, start: int = 0, out=None, stream=None):
    """Q, or (Q, K), [B, H, N, d] with any strides between rows, turned to their
    positions: positions[b, n] (int32, [N] or [B, N]) or start + n.  Returns new
    contiguous tensors, or writes ``out``, which may be the inputs themselves and lies
    otherwise apart from them (rows that interleave with its input's are refused)."""
    X, Y = _pair(Q, K, out)
    got = _rotate(rp, X, Y, positions, start, 0, stream)
    return got[0] if K is None else got


def rotary_bwd(rp: RotaryPlan, dQ, dK=None, positions=None, start: int = 0, out=None, stream=None):
    """Gradients of ``rotary``'s inputs from those of its outputs: the transposed map."""
    X, Y = _pair(dQ, dK, out)
    got = _rotate(rp, X, Y, positions, start, 1, stream)
    return got[0] if dK is None else got


# --- paged key-value cache ------------------------------------------------------


class PagedCache:
    """Keys and values of many sequences in pages: ``k`` and ``v``, [pages, H, page, d].

    A sequence is a row of a page table ([B, width] int32) and a length
    ([B] int32), both on the device and kept by the caller; slot j of sequence
    b is row j % page of page table[b, j // page].  Rows behind a length are
    never read."""

    def __init__(self, pages: int, page: int, H: int, d: int = 64, dtype: str = "bf16", device="cuda"):
        shape = (pages, H, page, d)
        self._set(*(torch.empty(shape, dtype=TORCH_DTYPE[DTYPES[dtype]], device=device) for _ in range(2)))

    @classmethod
    def of(cls, k, v):
        """A cache over existing tensors."""
        self = cls.__new__(cls)
        self._set(k, v)
        return self

    def _set(self, k, v):
        if not isinstance(k, torch.Tensor) or k.dim() != 4:
            raise ValueError("k: expected a tensor of shape [pages, H, page, d]")
        if k.dtype not in (torch.bfloat16, torch.float32):
            raise ValueError(f"k: dtype {k.dtype}, expected torch.bfloat16 or torch.float32")
        _rows_of(v, "v", k.dtype, *k.shape)
        for name, t in (("k", k), ("v", v)):
            if not t.is_contiguous():
                raise ValueError(f"{name}: must be contiguous")
        if v.device != k.device:
            raise ValueError(f"v: on {v.device}, k on {k.device}")
        if any(n >> 31 for n in k.shape[1:]):
            raise ValueError(f"k: shape {tuple(k.shape)}, expected H, page and d below 2^31")
        self._k, self._v = k, v
        self.pages, self.H, self.page, self.d = k.shape
        self._c = _PAGES(k.data_ptr(), v.data_ptr(), *k.shape, _dtype_code(k))
        self._needs = {}  # bytes of scratch by the sizes of a call

    @property
    def k(self):
        return self._k

    @property
    def v(self):
        return self._v

    @property
    def dtype(self):
        return self._k.dtype

    def _need(self, function, where, raw, B, capacity, *sizes):
        """function(raw, *sizes), remembered: it follows from the sizes alone."""
        key = (where, B, capacity, *sizes)
        n = self._needs.get(key)
        if n is None:
            n = function(raw, *sizes)
            if n < 0:
                if B:
                    _check(LIB.lh_last_status(), where)
                return 0
            if len(self._needs) > 256:
                self._needs.clear()
            self._needs[key] = n
        return n

    def _raw(self, table, lengths):
        """The lh_cache of one batch's table and lengths, B and the capacity."""
        if not isinstance(table, torch.Tensor) or table.dim() != 2:
            raise ValueError("table: expected a tensor of shape [B, width]")
        if table.dtype != torch.int32:
            raise ValueError(f"table: dtype {table.dtype}, expected torch.int32")
        B, width = table.shape
        if width > 1 and table.stride(1) != 1:
            raise ValueError("table: a sequence's pages must be contiguous")
        _index(lengths, "lengths", (B,))
        if (B | width) >> 31:
            raise ValueError(f"table: shape {tuple(table.shape)}, expected sizes below 2^31")
        return self._c + _BATCH(table.data_ptr(), table.stride(0), B, width, lengths.data_ptr()), B, width * self.page


def cache_append(cache: PagedCache, table, lengths, K, V, Q=None, rotary: RotaryPlan | None = None,
                 positions=None, counts=None, slot_positions=None, out=None, stream=None):
    """Write the new rows K, V ([B, H, T, d], any strides between rows) into the cache.

    ``lengths`` already count the new rows: row t < counts[b] (default T) goes
    to slot lengths[b] - counts[b] + t, rows behind are padding.  With
    ``rotary`` the keys, and the queries Q ([B, Hq, T, d]), are turned at
    positions ([T] or [B, T] int32, default: the slot).  Returns the turned
    queries (padding rows zero), in ``out`` if given (which may be Q), or None.  ``slot_positions`` ([B, H,
    capacity] int32) receives the positions of the new slots."""
    if not isinstance(K, torch.Tensor) or K.dim() != 4:
        raise ValueError("K: expected a tensor of shape [B, H, T, d]")
    raw, B, capacity = cache._raw(table, lengths)
    T, H, d, k = K.shape[2], cache.H, cache.d, cache._k
    new_k, new_v = _ROW(*_rows_of(K, "K", k.dtype, B, H, T, d)), _ROW(*_rows_of(V, "V", k.dtype, B, H, T, d))
    q = to = None
    if Q is not None:
        q = _ROW(*_rows_of(Q, "Q", k.dtype, B, None, T, d))
        if out is not None:
            to = _ROW(*_rows_of(out, "out", k.dtype, B, Q.shape[1], T, d))
    elif out is not None:
        raise ValueError("out: given without Q")
    stride = 0 if positions is None else _positions(positions, B, T)
    if counts is not None:
        _index(counts, "counts", (B,))
    if slot_positions is not None:
        _index(slot_positions, "slot_positions", (B, cache.H, capacity))
    if rotary is not None and rotary.d != d:
        raise ValueError(f"rotary: for d = {rotary.d}, the cache has d = {d}")
    dev = k.device
    tensors = (k, cache._v, K, V, table, lengths, positions, counts, slot_positions, Q, out)
    _on_device(dev, "cache cache K V table lengths positions counts slot_positions Q out", tensors)

    def call(handle):
        qo, qo_rows = out, to
        if Q is not None and out is None:
            qo = _contiguous_like(Q)
            qo_rows = _ROW(*_dense_rows(qo))
        if T and B:
            _check(LIB.lh_cache_append(raw, None if rotary is None else ctypes.byref(rotary.raw), T, new_k, new_v, q,
                                       qo_rows, _ptr(positions), stride, _ptr(counts), _ptr(slot_positions), handle),
                   "lh_cache_append")
        return (qo,)

    return _run(dev, stream, tensors, call)[0]


def decode(cache: PagedCache, table, lengths, Q, scale: float | None = None, weights=None,
           weights_out=None, ws=None, stream=None):
    """Attention of one new token of each sequence, Q [B, Hq, 1, d], over its
    cache: (O [B, Hq, 1, d], lse [B, Hq, 1]).  Hq is a multiple of the cache's
    H; neighbouring query heads share a key head.  An empty sequence gives
    O = 0 and lse = -inf.  scale: default 1 / sqrt(d).  ``weights`` ([B, H,
    capacity] fp32): each slot's attention probability, summed over the query
    heads of its key head, is added to it, in place or into ``weights_out``.
    ws: a uint8 scratch tensor of decode_ws_bytes(); calls that overlap on the
    GPU need one each (default: a new one)."""
    raw, B, capacity = cache._raw(table, lengths)
    k = cache._k
    rows = _rows_of(Q, "Q", k.dtype, B, None, 1, cache.d)
    Hq = rows[4]
    if weights is None and weights_out is not None:
        raise ValueError("weights_out: given without weights")
    if weights is not None:
        if weights_out is None:
            weights_out = weights
        for name, t in (("weights", weights), ("weights_out", weights_out)):
            _slots(t, name, torch.float32, (B, cache.H, capacity))
    dev = k.device
    need = cache._need(LIB.lh_decode_ws_bytes, "lh_decode_ws_bytes", raw, B, capacity, Hq, 0 if weights is None else 1)
    if ws is not None:
        _require(ws, "ws", torch.uint8, need)
    tensors = (k, cache._v, table, lengths, Q, weights, weights_out, ws)
    _on_device(dev, "cache cache table lengths Q weights weights_out ws", tensors)

    def call(handle):
        o = _contiguous_like(Q)
        lse = Q.new_empty((B, Hq, 1), dtype=torch.float32)
        w = _scratch(table, need) if ws is None else ws
        if B:
            _check(LIB.lh_decode(raw, _ROW(*rows), cache.d ** -0.5 if scale is None else scale,
                                 _ptr(o), _ptr(lse), _ptr(weights), _ptr(weights_out), _ptr(w), w.nbytes,
                                 handle), "lh_decode")
        return o, lse

    return _run(dev, stream, tensors, call)


def _scratch(table, nbytes: int):
    """At least ``nbytes`` on the table's device (16-byte aligned, like every allocation)."""
    return table.new_empty(max(4, (nbytes + 3) // 4))


def _slots(t, name: str, dtype, shape):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor, got {type(t).__name__}")
    if t.dtype != dtype:
        raise ValueError(f"{name}: dtype {t.dtype}, expected {dtype}")
    if t.shape != shape:
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {list(shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")


def decode_ws_bytes(cache: PagedCache, table, lengths, Hq: int, with_weights: bool = False) -> int:
    """Bytes of scratch that ``decode`` needs for this batch."""
    return cache._need(LIB.lh_decode_ws_bytes, "lh_decode_ws_bytes", *cache._raw(table, lengths), Hq, int(with_weights))


def evict(cache: PagedCache, table, lengths, weights, budget: int, positions=None, protect=None,
          weights_out=None, positions_out=None, ws=None, stream=None):
    """Keep the ``budget`` rows of largest weight of every sequence and head
    (ties: the lower slot) and give up the others, moving keys and values
    within their pages; returns (lengths, weights, positions) of what is left.

    weights: [B, H, capacity] fp32, as ``decode`` sums them.  Rows at or above
    position protect[b] ([B] int32) are kept before all others; positions
    ([B, H, capacity] int32, default: the slot) say where rows stand once
    earlier evictions have moved them.  Kept rows at low slots stay, the others
    fill the slots given up, so the order of slots is not that of positions;
    behind the new length weights are 0 and positions -1.  weights_out and
    positions_out (default: new tensors) may be the inputs themselves.  No two
    sequences may share a page, for both would move its rows.  ws: a
    uint8 scratch tensor of evict_ws_bytes(); calls that overlap on the GPU
    need one each (default: a new one)."""
    raw, B, capacity = cache._raw(table, lengths)
    shape = (B, cache.H, capacity)
    _slots(weights, "weights", torch.float32, shape)
    if weights_out is not None:
        _slots(weights_out, "weights_out", torch.float32, shape)
    if positions is None and positions_out is not None:
        raise ValueError("positions_out: given without positions")
    for name, t in (("positions", positions), ("positions_out", positions_out)):
        if t is not None:
            _slots(t, name, torch.int32, shape)
    if protect is not None:
        _index(protect, "protect", (B,))
    dev = cache._k.device
    need = cache._need(LIB.lh_evict_ws_bytes, "lh_evict_ws_bytes", raw, B, capacity, budget)
    if ws is not None:
        _require(ws, "ws", torch.uint8, need)
    tensors = (cache._k, cache._v, table, lengths, weights, weights_out, positions, positions_out, protect, ws)
    _on_device(dev, "cache cache table lengths weights weights_out positions positions_out protect ws", tensors)

    def call(handle):
        n = torch.empty_like(lengths)
        wo = torch.empty_like(weights) if weights_out is None else weights_out
        po = torch.empty_like(positions) if positions is not None and positions_out is None else positions_out
        w = _scratch(table, need) if ws is None else ws
        if B:
            _check(LIB.lh_evict(raw, budget, _ptr(weights), _ptr(positions), _ptr(protect),
                                _ptr(wo), _ptr(po), _ptr(n), _ptr(w), w.nbytes, handle), "lh_evict")
        return n, wo, po

    return _run(dev, stream, tensors, call)


def evict_ws_bytes(cache: PagedCache, table, lengths, budget: int) -> int:
    """Bytes of scratch that ``evict`` needs for this batch."""
    return cache._need(LIB.lh_evict_ws_bytes, "lh_evict_ws_bytes", *cache._raw(table, lengths), budget)


# --- whole layer --------------------------------------------------------------


class Context:
    """The forward-to-backward buffer of one lh_forward call, with typed views."""

    def __init__(self, pl: Plan, device):
        self.plan = pl
        self.buf = _bytes(pl.raw.ctx_bytes, device)
        self.rotary = None  # (plan, positions, start) of the forward's Q and K

    def _view(self, off, shape, dtype):
        n = 1
        for s in shape:
            n *= s
        nbytes = n * torch.tensor([], dtype=dtype).element_size()
        return self.buf[off: off + nbytes].view(dtype).view(shape)

    @property
    def sel_idx(self):
        c = self.plan.raw.c
        return self._view(self.plan.raw.ctx_sel_idx, (c.B, c.H, self.plan.S), torch.int32)

    @property
    def slot_of(self):
        c = self.plan.raw.c
        return self._view(self.plan.raw.ctx_slot_of, (c.B, c.H, self.plan.Ntot), torch.int32)

    def gathered(self, name):
        c = self.plan.raw.c
        off = getattr(self.plan.raw, "ctx_" + name)
        return self._view(off, (c.B, c.H, self.plan.S, c.d), self.plan.dtype)

    @property
    def lse(self):
        c = self.plan.raw.c
        return self._view(self.plan.raw.ctx_lse, (c.B, c.H, self.plan.S), torch.float32)


class Workspace:
    def __init__(self, pl: Plan, device):
        self.buf = _bytes(pl.raw.ws_bytes, device)


def _bhnd(pl: Plan, *tensors):
    """[B, H, N, d] views of contiguous tensors of at least that many elements."""
    c = pl.raw.c
    return tuple(t.view(-1)[: c.B * c.H * c.N * c.d].view(c.B, c.H, c.N, c.d) for t in tensors)


def forward(pl: Plan, Q, K, V, O=None, ctx: Context | None = None, ws: Workspace | None = None,
            stream=None, rotary: RotaryPlan | None = None, positions=None, start: int = 0):
    """O = Lighthouse(Q, K, V); returns (O, ctx).  With ``rotary`` the layer
    runs on Q and K turned to their positions (copies, as ``lh.rotary`` makes
    them), and the matching ``backward`` turns their gradients back; positions
    must not change in between."""
    if rotary is None and (positions is not None or start != 0):
        raise ValueError("positions, start: given without rotary")
    _require_tokens(pl, Q=Q, K=K, V=V)
    dev = Q.device
    if O is None:
        O = torch.empty_like(Q)
    if rotary is not None:
        Q, K = _rotate(rotary, _bhnd(pl, Q, K), None, positions, start, 0, stream)
    if ctx is None:
        ctx = Context(pl, dev)
    if ws is None:
        ws = Workspace(pl, dev)
    _require_tokens(pl, O=O)
    _require(ctx.buf, "ctx", torch.uint8, pl.raw.ctx_bytes)
    _require(ws.buf, "ws", torch.uint8, pl.raw.ws_bytes)
    _check(LIB.lh_forward(pl.byref(), _ptr(Q), _ptr(K), _ptr(V), _ptr(O), _ptr(ctx.buf),
                          ctx.buf.numel(), _ptr(ws.buf), ws.buf.numel(), _stream(stream)),
           "lh_forward")
    ctx.rotary = None if rotary is None else (rotary, positions, start)
    return O, ctx


def backward(pl: Plan, dO, ctx: Context, dQ=None, dK=None, dV=None, ws: Workspace | None = None,
             stream=None):
    """(dQ, dK, dV) from dO and the ctx of the matching forward."""
    _require_tokens(pl, dO=dO)
    if dQ is None:
        dQ, dK, dV = torch.empty_like(dO), torch.empty_like(dO), torch.empty_like(dO)
    if ws is None:
        ws = Workspace(pl, dO.device)
    _require_tokens(pl, dQ=dQ, dK=dK, dV=dV)
    _require(ctx.buf, "ctx", torch.uint8, pl.raw.ctx_bytes)
    _require(ws.buf, "ws", torch.uint8, pl.raw.ws_bytes)
    _check(LIB.lh_backward(pl.byref(), _ptr(dO), _ptr(ctx.buf), ctx.buf.numel(), _ptr(dQ),
                           _ptr(dK), _ptr(dV), _ptr(ws.buf), ws.buf.numel(), _stream(stream)),
           "lh_backward")
    if ctx.rotary is not None:
        rp, positions, start = ctx.rotary
        grads = _bhnd(pl, dQ, dK)
        _rotate(rp, grads, grads, positions, start, 1, stream)
    return dQ, dK, dV


class HostPipeline:
    """Forward and backward of one layer per step on host (pinned) tensors.

    Each step copies Q, K, V, dO to the device, runs lh_forward and
    lh_backward, and copies O, dQ, dK, dV back.  Two device buffer sets and
    three streams let the copy-in of step i+1 and the copy-out of step i-1
    run while the kernels of step i do (PCIe is full duplex; the kernels use
    only the compute stream).  ``step`` enqueues and returns at once;
    ``synchronize`` waits for every enqueued step.  The host tensors passed to
    a step must stay untouched until it has completed.
    """

    def __init__(self, pl: Plan, device):
        c = pl.raw.c
        shape = (c.B, c.H, c.N, c.d)
        self.pl = pl
        self.inputs = [[torch.empty(shape, dtype=pl.dtype, device=device) for _ in range(4)]
                       for _ in range(2)]
        self.outputs = [[torch.empty(shape, dtype=pl.dtype, device=device) for _ in range(4)]
                        for _ in range(2)]
        self.ctx = Context(pl, device)
        self.ws = Workspace(pl, device)
        self.s_in, self.s_run, self.s_out = (torch.cuda.Stream(device) for _ in range(3))
        self.copied_in = [torch.cuda.Event() for _ in range(2)]
        self.done = [torch.cuda.Event() for _ in range(2)]
        self.copied_out = [torch.cuda.Event() for _ in range(2)]
        self.used = [False, False]
        self.n = 0

    def step(self, host_inputs, host_outputs):
        """host_inputs: (Q, K, V, dO); host_outputs: (O, dQ, dK, dV); pinned, [B,H,N,d]."""
        b = self.n % 2
        self.n += 1
        dev_in, dev_out = self.inputs[b], self.outputs[b]
        if self.used[b]:  # this buffer set's previous step has read its inputs
            self.s_in.wait_event(self.done[b])
        with torch.cuda.stream(self.s_in):
            for d, h in zip(dev_in, host_inputs):
                d.copy_(h, non_blocking=True)
            self.copied_in[b].record(self.s_in)
        self.s_run.wait_event(self.copied_in[b])
        if self.used[b]:  # and its outputs have left the device
            self.s_run.wait_event(self.copied_out[b])
        Q, K, V, dO = dev_in
        O, dQ, dK, dV = dev_out
        forward(self.pl, Q, K, V, O, self.ctx, self.ws, stream=self.s_run)
        backward(self.pl, dO, self.ctx, dQ, dK, dV, self.ws, stream=self.s_run)
        self.done[b].record(self.s_run)
        self.s_out.wait_event(self.done[b])
        with torch.cuda.stream(self.s_out):
            for h, d in zip(host_outputs, dev_out):
                h.copy_(d, non_blocking=True)
            self.copied_out[b].record(self.s_out)
        self.used[b] = True

    def wait_on(self, event):
        """Make every stream of the pipeline wait for `event` (e.g. a start marker)."""
        for st in (self.s_in, self.s_run, self.s_out):
            st.wait_event(event)

    def record_end(self, stream):
        """Make `stream` wait for everything enqueued so far."""
        for ev in self.copied_in + self.done + self.copied_out:
            stream.wait_event(ev)

    def synchronize(self):
        for st in (self.s_in, self.s_run, self.s_out):
            st.synchronize()


def set_deterministic(on: bool):
    """Process-wide: bit-reproducible bf16 attention backward (two kernels, no
    atomics) for lh_attn_bwd / lh_backward calls enqueued afterwards."""
    LIB.lh_set_deterministic(1 if on else 0)


def selftest_wait_timeout(stream=None):
    """Enqueue the failure-path self-test (a bounded wait that must give up);
    the next device_status() raises LighthouseError with LH_ERR_TIMEOUT."""
    _check(LIB.lh_selftest_wait_timeout(_stream(stream)), "lh_selftest_wait_timeout")


def device_status(reset: bool = True):
    _check(LIB.lh_device_status(1 if reset else 0), "lh_device_status")
