"""Log-linear Sparse Attention (LLSA) for GB300 (sm_103a): Python binding.

A thin ctypes layer over the C ABI of ``include/llsa.h`` (libllsa.so, built
in-tree by ``build.build()``). The functions keep the C names -- ``llsa_pool``,
``llsa_select``, ``llsa_fwd``, ``llsa_index_transpose``, ``llsa_bwd`` -- and do
argument marshalling only: every step of the computation runs in the
library's CUDA kernels on the caller's current torch stream. PyTorch supplies
device memory and streams. There is no CPU fallback: if the library is not
built or the device is not a GB300, calls raise.

Beside the sparse path: dense attention (``llsa_dense_fwd``, ``llsa_dense_bwd``;
``dense_attention`` with autograd), differential attention (``llsa_diff_fwd``,
``llsa_diff_bwd``; ``diff_attention`` with autograd) and rotary positions on one or two axes
(``llsa_rope``) or up to four (``llsa_rope_grid``): ``rotary``, or ``rope=`` of any
attention.

Method: "Trainable Log-linear Sparse Attention for Efficient Diffusion
Transformers" (arXiv 2512.16615), as described on its Pith review page
("Core claim", "What carries the argument").
"""
from __future__ import annotations

import contextlib
import ctypes
import functools
import math
import os
from dataclasses import dataclass, replace

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(_PKG, "_build", "libllsa.so")
_lib = None

LLSA_DTYPE_BF16, LLSA_DTYPE_F32 = 0, 1
LLSA_ENRICH_TOP1 = 0
LLSA_ENRICH_ANCESTOR = 1
LLSA_ENRICH_ALLK = 2
_RULES = {"top1": LLSA_ENRICH_TOP1, "ancestor": LLSA_ENRICH_ANCESTOR, "allk": LLSA_ENRICH_ALLK}
LLSA_ORDER_TILE, LLSA_ORDER_RASTER = 0, 1
_ORDERS = {"tile": LLSA_ORDER_TILE, "raster": LLSA_ORDER_RASTER}
OP_POOL, OP_SELECT, OP_FWD, OP_TRANSPOSE, OP_BWD, OP_DENSE_FWD, OP_DENSE_BWD, OP_DIFF_FWD, OP_DIFF_BWD = range(9)
LLSA_ROPE_HALF, LLSA_ROPE_INTERLEAVED = 0, 1
_ROPE_LAYOUTS = {"half": LLSA_ROPE_HALF, "interleaved": LLSA_ROPE_INTERLEAVED}
_ROPE_SCALINGS = {"none": 0, "linear": 1, "base": 2, "wavelength": 3}
LLSA_ROPE_SPAN_AXIS, LLSA_ROPE_SPAN_HEAD, LLSA_ROPE_SPAN_DEALT = 0, 1, 2
_ROPE_SPANS = {"axis": LLSA_ROPE_SPAN_AXIS, "head": LLSA_ROPE_SPAN_HEAD, "dealt": LLSA_ROPE_SPAN_DEALT}
ROPE_MAX_AXES = 4
MAX_LEVELS = 8


class LLSAError(RuntimeError):
    """A negative LLSA_* status from the library."""

    def __init__(self, code: int, where: str):
        self.code = code
        super().__init__(f"{where}: {strerror(code)} (code {code})")


class _Params(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int), ("heads", ctypes.c_int), ("n", ctypes.c_int), ("d", ctypes.c_int),
                ("block", ctypes.c_int), ("levels", ctypes.c_int), ("topk", ctypes.c_int),
                ("enrich_levels", ctypes.c_int), ("dtype", ctypes.c_int), ("scale", ctypes.c_float),
                ("enrich_rule", ctypes.c_int), ("token_order", ctypes.c_int)]


class _Sizes(ctypes.Structure):
    _fields_ = [("levels", ctypes.c_int), ("enrich_levels", ctypes.c_int),
                ("n_level", ctypes.c_int * (MAX_LEVELS + 1)), ("topk_level", ctypes.c_int * (MAX_LEVELS + 1)),
                ("row_offset", ctypes.c_int * (MAX_LEVELS + 1)), ("pyr_rows", ctypes.c_int),
                ("n_blocks", ctypes.c_int), ("keys_per_query", ctypes.c_int), ("slices", ctypes.c_longlong),
                ("level_idx_offset", ctypes.c_longlong * (MAX_LEVELS + 1)),
                ("level_idx_per_slice", ctypes.c_longlong), ("scale", ctypes.c_float),
                ("coarse_cols", ctypes.c_int), ("enrich_cols", ctypes.c_int)]


class _DenseParams(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in ("batch", "heads", "kv_heads", "nq", "nk", "d", "dtype", "causal")] + [
        ("scale", ctypes.c_float)]


class _DiffParams(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in ("batch", "heads", "kv_heads", "nq", "nk", "d", "dtype", "lam_dtype", "qk_fp32", "causal")] + [
        ("scale", ctypes.c_float)]


class _RopeParams(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in ("batch", "heads", "kv_heads", "n", "d", "rot_dim", "layout", "axes", "width",
                                            "token_order", "pos_offset", "pos_batched", "dtype", "scaling", "orig_len")] + [
        (n, ctypes.c_double) for n in ("base", "factor", "low", "high", "amplitude")]


class _RopeStrides(ctypes.Structure):
    _fields_ = [(n, ctypes.c_longlong * 3) for n in ("q", "k", "q_out", "k_out")]


class _RopeGridParams(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in ("batch", "heads", "kv_heads", "n", "d", "layout", "span", "axes")] + [
        (n, ctypes.c_int * ROPE_MAX_AXES) for n in ("columns", "extent", "offset")] + [
        (n, ctypes.c_int) for n in ("token_order", "pos_batched", "dtype", "out_other", "scaling", "orig_len")] + [
        (n, ctypes.c_double) for n in ("base", "factor", "low", "high", "amplitude")] + [("step", ctypes.c_double * ROPE_MAX_AXES)]


def lib_path() -> str:
    return _LIB_PATH


def _load():
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(_LIB_PATH):
        raise RuntimeError(f"LLSA CUDA library not built ({_LIB_PATH}); run "
                           "hierarchical_sparse_attention_mean_gb300.build.build()")
    lib = ctypes.CDLL(_LIB_PATH)
    P = ctypes.POINTER(_Params)
    vp, sz = ctypes.c_void_p, ctypes.c_size_t
    lib.llsa_get_sizes.argtypes = [P, ctypes.POINTER(_Sizes)]
    lib.llsa_workspace_bytes.argtypes = [P, ctypes.c_int]
    lib.llsa_workspace_bytes.restype = sz
    lib.llsa_pool.argtypes = [P, vp, vp, vp, vp, vp, sz, vp]
    lib.llsa_select.argtypes = [P, vp, vp, vp, vp, vp, sz, vp]
    lib.llsa_fwd.argtypes = [P, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    lib.llsa_index_transpose.argtypes = [P, vp, vp, vp, vp, sz, vp]
    lib.llsa_reorder.argtypes = [P, ctypes.c_int, ctypes.c_int, vp, vp, ctypes.c_int, vp]
    lib.llsa_select_exhaustive.argtypes = [P, vp, vp, vp]
    lib.llsa_bwd.argtypes = [P] + [vp] * 14 + [vp, sz, vp]
    DP = ctypes.POINTER(_DenseParams)
    lib.llsa_dense_workspace_bytes.argtypes = [DP, ctypes.c_int]
    lib.llsa_dense_workspace_bytes.restype = sz
    lib.llsa_dense_fwd.argtypes = [DP] + [vp] * 8 + [sz, vp]
    lib.llsa_dense_bwd.argtypes = [DP] + [vp] * 12 + [sz, vp]
    FP = ctypes.POINTER(_DiffParams)
    lib.llsa_diff_workspace_bytes.argtypes = [FP, ctypes.c_int]
    lib.llsa_diff_workspace_bytes.restype = sz
    lib.llsa_diff_fwd.argtypes = [FP] + [vp] * 10 + [sz, vp]
    lib.llsa_diff_bwd.argtypes = [FP] + [vp] * 15 + [sz, vp]
    lib.llsa_rope.argtypes = [ctypes.POINTER(_RopeParams), ctypes.POINTER(_RopeStrides)] + [vp] * 5 + [ctypes.c_int, vp]
    lib.llsa_rope_grid.argtypes = [ctypes.POINTER(_RopeGridParams), ctypes.POINTER(_RopeStrides)] + [vp] * 5 + [ctypes.c_int, vp]
    lib.llsa_get_status.argtypes = [vp, ctypes.POINTER(ctypes.c_int)]
    lib.llsa_strerror.argtypes = [ctypes.c_int]
    lib.llsa_strerror.restype = ctypes.c_char_p
    lib.llsa_launch_count.restype = ctypes.c_ulonglong
    lib.llsa_test_set_wait_limit.argtypes = [ctypes.c_int, ctypes.c_int]
    lib.llsa_profile_enable.argtypes = [ctypes.c_int]
    lib.llsa_profile_only.argtypes = [ctypes.c_char_p]
    lib.llsa_profile_read.argtypes = [ctypes.POINTER(ctypes.c_char_p), ctypes.POINTER(ctypes.c_float), ctypes.c_int]
    _lib = lib
    return lib


def strerror(code: int) -> str:
    return _load().llsa_strerror(code).decode()


def _check(rc: int, where: str):
    if rc != 0:
        raise LLSAError(rc, where)


@dataclass(frozen=True)
class Params:
    """Problem description; mirrors llsa_params of include/llsa.h."""
    batch: int
    heads: int
    n: int
    d: int
    block: int = 16
    topk: int = 8
    levels: int = 0            # 0: floor(log_B n - 1)
    enrich_levels: int = -1    # -1: all levels; 0: no enrichment
    dtype: str = "bf16"        # "bf16" or "fp32"
    scale: float = 0.0         # 0: 1/sqrt(d)
    enrich_rule: str = "top1"  # "top1", "ancestor" or "allk"
    token_order: str = "tile"  # "tile" or "raster" (raster order of a square image)

    def c(self) -> _Params:
        dt = {"bf16": LLSA_DTYPE_BF16, "fp32": LLSA_DTYPE_F32}.get(self.dtype)
        if dt is None:
            raise ValueError(f"dtype must be 'bf16' or 'fp32', not {self.dtype!r}")
        rule = _RULES.get(self.enrich_rule)
        if rule is None:
            raise ValueError(f"enrich_rule must be 'top1', 'ancestor' or 'allk', not {self.enrich_rule!r}")
        order = _ORDERS.get(self.token_order)
        if order is None:
            raise ValueError(f"token_order must be 'tile' or 'raster', not {self.token_order!r}")
        return _Params(self.batch, self.heads, self.n, self.d, self.block, self.levels, self.topk,
                       self.enrich_levels, dt, self.scale, rule, order)

    @staticmethod
    def like(q, **kw) -> "Params":
        b, h, n, d = q.shape
        dtype = {torch.bfloat16: "bf16", torch.float32: "fp32"}.get(q.dtype)
        if dtype is None:
            raise ValueError("q must be bfloat16 or float32")
        return Params(b, h, n, d, dtype=dtype, **kw)


_DTYPES = {"bf16": LLSA_DTYPE_BF16, "fp32": LLSA_DTYPE_F32}


def _choice(table, value, name):
    got = table.get(value)
    if got is None:
        raise ValueError(f"{name} must be one of {', '.join(map(repr, table))}, not {value!r}")
    return got


def _dtype_name(t, what="q"):
    name = {torch.bfloat16: "bf16", torch.float32: "fp32"}.get(t.dtype)
    if name is None:
        raise ValueError(f"{what} must be bfloat16 or float32")
    return name


def _int32(**fields):
    """Refuses what a C int would cut to its low bits."""
    for name, value in fields.items():
        if not -(1 << 31) <= value < 1 << 31:
            raise ValueError(f"{name} must fit 32 bits, not {value}")


@dataclass(frozen=True)
class DenseParams:
    """A dense-attention problem; mirrors llsa_dense_params of include/llsa.h."""
    batch: int
    heads: int
    nq: int
    nk: int
    d: int
    kv_heads: int = 0          # 0: as many as heads
    causal: bool = False       # the last query sees the last key
    dtype: str = "bf16"        # "bf16" or "fp32"
    scale: float = 0.0         # 0: 1/sqrt(d)

    def __post_init__(self):
        self.__dict__.update(_dense_native(self.batch, self.heads, self.nq, self.nk, self.d, self.kv_heads, bool(self.causal),
                                           self.dtype, float(self.scale)))

    def __reduce__(self):  # copies and pickles build their own C structure
        return DenseParams, (self.batch, self.heads, self.nq, self.nk, self.d, self.kv_heads, self.causal, self.dtype,
                             self.scale)

    def c(self) -> _DenseParams:
        return self._c

    @staticmethod
    def like(q, k, causal: bool = False, scale: float = 0.0) -> "DenseParams":
        """The parameters of a call on q and k (equal calls share one object)."""
        return _dense_params(tuple(q.shape), tuple(k.shape), _dtype_name(q), bool(causal), float(scale))

    def shapes(self):
        """Shapes of q (and o, dout, dq), of k (and v, dk, dv) and of lse."""
        return self._shapes


@functools.lru_cache(maxsize=256)
def _dense_native(batch, heads, nq, nk, d, kv_heads, causal, dtype, scale):
    """What equal parameters share: the C structure, the workspace sizes, the tensors' shapes."""
    _int32(batch=batch, heads=heads, kv_heads=kv_heads, nq=nq, nk=nk, d=d)
    c = _DenseParams(batch, heads, kv_heads, nq, nk, d, _choice(_DTYPES, dtype, "dtype"), 1 if causal else 0, scale)
    return {"_c": c, "_ref": ctypes.byref(c), "_ws": {},
            "_shapes": ((batch, heads, nq, d), (batch, kv_heads or heads, nk, d), (batch, heads, nq))}


@functools.lru_cache(maxsize=256)
def _dense_params(q, k, dtype, causal, scale):
    b, h, n, d = q
    return DenseParams(b, h, n, k[2], d, kv_heads=k[1], causal=causal, dtype=dtype, scale=scale)


@dataclass(frozen=True)
class DiffParams:
    """A differential-attention problem; mirrors llsa_diff_params of include/llsa.h."""
    batch: int
    heads: int                 # differential heads: q has twice as many
    nq: int
    nk: int
    d: int                     # columns of q and k; v and o have twice as many
    kv_heads: int = 0          # value heads, and key heads of each map; 0: as many as heads
    causal: bool = False       # the last query sees the last key
    dtype: str = "bf16"        # "bf16" or "fp32"
    lam_dtype: str = ""        # of lam and its gradient; "": dtype
    scale: float = 0.0         # 0: 1/sqrt(d)
    qk_dtype: str = ""         # of q, k, their gradients and o2; "": dtype, else "fp32"

    def __post_init__(self):
        self.__dict__.update(_diff_native(self.batch, self.heads, self.nq, self.nk, self.d, self.kv_heads, bool(self.causal),
                                          self.dtype, self.lam_dtype or self.dtype, float(self.scale), self.qk_dtype or self.dtype))

    def __reduce__(self):  # copies and pickles build their own C structure
        return DiffParams, (self.batch, self.heads, self.nq, self.nk, self.d, self.kv_heads, self.causal, self.dtype,
                            self.lam_dtype, self.scale, self.qk_dtype)

    def c(self) -> _DiffParams:
        return self._c

    @staticmethod
    def like(q, k, lam=None, causal: bool = False, scale: float = 0.0, v=None) -> "DiffParams":
        """The parameters of a call on q, k and lam (equal calls share one object); with v, its type
        may be another than q's."""
        return _diff_params(tuple(q.shape), tuple(k.shape), _dtype_name(q), "" if lam is None else _dtype_name(lam, "lam"),
                            bool(causal), float(scale), _dtype_name(q if v is None else v))

    def shapes(self):
        """Shapes of q (and dq), of k (and dk), of v (and dv), of o (and o2, dout) and of lse."""
        return self._shapes


@functools.lru_cache(maxsize=256)
def _diff_native(batch, heads, nq, nk, d, kv_heads, causal, dtype, lam_dtype, scale, qk_dtype):
    """What equal parameters share: the C structure, the workspace sizes, the tensors' shapes."""
    _int32(batch=batch, heads=heads, kv_heads=kv_heads, nq=nq, nk=nk, d=d)
    if qk_dtype != dtype and qk_dtype != "fp32":
        raise ValueError(f"qk_dtype must be dtype or 'fp32', not {qk_dtype!r}")
    c = _DiffParams(batch, heads, kv_heads, nq, nk, d, _choice(_DTYPES, dtype, "dtype"), _choice(_DTYPES, lam_dtype, "lam_dtype"),
                    1 if qk_dtype != dtype else 0, 1 if causal else 0, scale)
    kv = kv_heads or heads
    types = {"bf16": torch.bfloat16, "fp32": torch.float32}
    shapes = ((batch, 2 * heads, nq, d), (batch, 2 * kv, nk, d), (batch, kv, nk, 2 * d), (batch, heads, nq, 2 * d), (batch, 2 * heads, nq))
    (sq, sk, sv, so, sl), td, qk = shapes, types[dtype], types[qk_dtype]
    given = (("q", qk, sq), ("k", qk, sk), ("v", td, sv), ("lam", types[lam_dtype], (heads,)))
    o, o2, lse = ("o", td, so), ("o2", qk, so), ("lse", torch.float32, sl)
    return {"_c": c, "_ref": ctypes.byref(c), "_ws": {}, "_shapes": shapes, "_fwd": (*given, o, lse, o2),
            "_bwd": (*given, o, o2, lse, ("dout", td, so), *(("d" + name, t, x) for name, t, x in given))}


@functools.lru_cache(maxsize=256)
def _diff_params(q, k, qk_dtype, lam_dtype, causal, scale, dtype):
    b, h, n, d = q
    if h % 2 or k[1] % 2:
        raise ValueError(f"q and k must have two heads for each differential one, got {h} and {k[1]}")
    return DiffParams(b, h // 2, n, k[2], d, kv_heads=k[1] // 2, causal=causal, dtype=dtype, lam_dtype=lam_dtype, scale=scale,
                      qk_dtype=qk_dtype)


@dataclass(frozen=True)
class RopeParams:
    """Rotary positions of q and k; mirrors llsa_rope_params of include/llsa.h."""
    batch: int
    heads: int
    n: int
    d: int
    kv_heads: int = 0            # heads of k; 0: no k
    rot_dim: int = 0             # columns turned; 0: d
    layout: str = "half"         # pairs: "half" (i, i + h) or "interleaved" (2i, 2i + 1)
    axes: int = 1                # 1, or 2 (row and column, half of the columns each)
    width: int = 0               # image width (axes 2; ignored with pos)
    token_order: str = "raster"  # "raster" or "tile" (axes 2; ignored with pos)
    pos_offset: int = 0          # position of token 0 (axes 1; ignored with pos)
    base: float = 10000.0
    scaling: str = "none"        # "none", "linear", "base" or "wavelength"
    factor: float = 1.0
    orig_len: int = 0            # "wavelength": positions the model was trained on
    low: float = 1.0             # "wavelength": turns over orig_len below which a pair is stretched fully
    high: float = 32.0           # and above which it is kept
    amplitude: float = 0.0       # 0: 1, or 0.1 ln(factor) + 1 for "wavelength" with a factor above 1
    dtype: str = "bf16"

    def __post_init__(self):
        self.__dict__["_c"] = _rope_native(
            self.batch, self.heads, self.kv_heads, self.n, self.d, self.rot_dim, self.layout, self.axes, self.width,
            self.token_order, self.pos_offset, self.dtype, self.scaling, self.orig_len, float(self.base), float(self.factor),
            float(self.low), float(self.high), float(self.amplitude))

    def c(self, pos_batched: bool = False) -> _RopeParams:
        return self._c[1 if pos_batched else 0]

    def grid(self, has_pos: bool = False) -> "RopeGridParams | None":
        """The same positions as parameters of llsa_rope_grid; None where it has none (an image whose
        last row is not full, fields that llsa_rope refuses)."""
        got = self.__dict__.get("_grid", {}).get(has_pos, self)
        if got is not self:
            return got
        rot = self.rot_dim or self.d
        if has_pos:
            extent = None
        elif self.axes == 1:
            extent = (self.n,)
        else:
            extent = (self.n // self.width, self.width) if self.width > 0 and self.n % self.width == 0 else 0
        stray = not has_pos and (self.width if self.axes == 1 else self.pos_offset)  # a field of the other kind of axes
        if self.axes not in (1, 2) or extent == 0 or stray or rot % (2 * self.axes):
            got = None
        else:
            got = RopeGridParams(self.batch, self.heads, self.n, self.d, kv_heads=self.kv_heads, columns=(rot // self.axes,) * self.axes,
                                 extent=extent, offset=() if self.axes == 2 or has_pos else (self.pos_offset,), layout=self.layout,
                                 token_order=self.token_order if self.axes == 2 else "raster", base=self.base, scaling=self.scaling,
                                 factor=self.factor, orig_len=self.orig_len, low=self.low, high=self.high, amplitude=self.amplitude,
                                 dtype=self.dtype)
        self.__dict__.setdefault("_grid", {})[has_pos] = got
        return got

    def in_fp32(self) -> "RopeParams":
        """The same positions for fp32 tensors."""
        got = self.__dict__.get("_fp32")
        if got is None:
            got = self.__dict__["_fp32"] = replace(self, dtype="fp32")
        return got

    @staticmethod
    def like(q, k=None, **kw) -> "RopeParams":
        b, h, n, d = q.shape
        return RopeParams(b, h, n, d, kv_heads=0 if k is None else k.shape[1], dtype=_dtype_name(q), **kw)


@functools.lru_cache(maxsize=256)
def _rope_native(batch, heads, kv_heads, n, d, rot_dim, layout, axes, width, order, offset, dtype, scaling, orig_len, *real):
    """The C structures of equal parameters, for positions without and with a batch dimension."""
    _int32(batch=batch, heads=heads, kv_heads=kv_heads, n=n, d=d, rot_dim=rot_dim, axes=axes, width=width, pos_offset=offset,
           orig_len=orig_len)
    layout, order = _choice(_ROPE_LAYOUTS, layout, "layout"), _choice(_ORDERS, order, "token_order")
    dtype, scaling = _choice(_DTYPES, dtype, "dtype"), _choice(_ROPE_SCALINGS, scaling, "scaling")
    return tuple(_RopeParams(batch, heads, kv_heads, n, d, rot_dim, layout, axes, width, order, offset, batched, dtype,
                             scaling, orig_len, *real) for batched in (0, 1))


@dataclass(frozen=True)
class RopeGridParams:
    """Rotary positions on up to four axes; mirrors llsa_rope_grid_params of include/llsa.h.

    The tokens are a grid of `extent` entries, the last axis fastest, or have their
    positions in `pos` (extent None)."""
    batch: int
    heads: int
    n: int
    d: int
    kv_heads: int = 0            # heads of k; 0: no k
    columns: tuple = ()          # columns turned by each axis; one entry per axis
    extent: tuple | None = None  # entries of the grid on each axis; None: positions are given
    offset: tuple = ()           # position of the grid's first entry on each axis; (): 0
    step: tuple = ()             # positions per entry on each axis; (): 1
    span: str = "axis"           # frequencies: a ladder per "axis", one over the "head", or that one "dealt" in turn
    layout: str = "half"         # pairs: "half" (i, i + h) or "interleaved" (2i, 2i + 1)
    token_order: str = "raster"  # "raster", or "tile": the last two axes are a frame in tile order
    base: float = 10000.0
    scaling: str = "none"        # "none", "linear", "base" or "wavelength"
    factor: float = 1.0
    orig_len: int = 0            # "wavelength": positions the model was trained on
    low: float = 1.0             # "wavelength": as RopeParams
    high: float = 32.0
    amplitude: float = 0.0       # 0: 1, or 0.1 ln(factor) + 1 for "wavelength" with a factor above 1
    dtype: str = "bf16"
    out_dtype: str = ""          # of q_out and k_out; "": dtype

    def __post_init__(self):
        for name in ("columns", "extent", "offset", "step"):
            value = getattr(self, name)
            if value is not None:
                self.__dict__[name] = tuple(value)
        axes = len(self.columns)
        if not 1 <= axes <= ROPE_MAX_AXES:
            raise ValueError(f"columns must have 1 to {ROPE_MAX_AXES} entries, one per axis, not {axes}")
        for name in ("extent", "offset", "step"):
            value = getattr(self, name)
            if value and len(value) != axes:
                raise ValueError(f"{name} must have an entry for each of the {axes} axes, not {len(value)}")
        self.__dict__["_c"] = _rope_grid_native(
            self.batch, self.heads, self.kv_heads, self.n, self.d, self.columns, self.extent or (), self.offset,
            tuple(float(x) for x in self.step), self.span, self.layout, self.token_order, self.dtype, self.out_dtype or self.dtype,
            self.scaling, self.orig_len, float(self.base), float(self.factor), float(self.low), float(self.high),
            float(self.amplitude))

    @property
    def axes(self) -> int:
        return len(self.columns)

    def c(self, pos_batched: bool = False) -> _RopeGridParams:
        return self._c[1 if pos_batched else 0]

    def in_fp32(self) -> "RopeGridParams":
        """The same positions for fp32 tensors."""
        return self._kept("_fp32", dtype="fp32", out_dtype="")

    def to_fp32(self) -> "RopeGridParams":
        """The same positions, from bf16 into fp32."""
        return self._kept("_up", dtype="bf16", out_dtype="fp32")

    def from_fp32(self) -> "RopeGridParams":
        """The same positions, from fp32 into bf16."""
        return self._kept("_down", dtype="fp32", out_dtype="bf16")

    def _kept(self, name, **kw):
        got = self.__dict__.get(name)
        if got is None:
            got = self.__dict__[name] = replace(self, **kw)
        return got

    def grid(self, has_pos: bool = False) -> "RopeGridParams":
        return self

    @staticmethod
    def like(q, k=None, **kw) -> "RopeGridParams":
        b, h, n, d = q.shape
        return RopeGridParams(b, h, n, d, kv_heads=0 if k is None else k.shape[1], dtype=_dtype_name(q), **kw)


@functools.lru_cache(maxsize=256)
def _rope_grid_native(batch, heads, kv_heads, n, d, columns, extent, offset, step, span, layout, order, dtype, out_dtype, scaling,
                      orig_len, *real):
    """The C structures of equal parameters, for positions without and with a batch dimension."""
    _int32(batch=batch, heads=heads, kv_heads=kv_heads, n=n, d=d, orig_len=orig_len)
    for name, values in (("columns", columns), ("extent", extent), ("offset", offset)):
        for value in values:
            _int32(**{name: value})
    four = [(ctypes.c_int * ROPE_MAX_AXES)(*x) for x in (columns, extent, offset)]
    span, layout = _choice(_ROPE_SPANS, span, "span"), _choice(_ROPE_LAYOUTS, layout, "layout")
    order = _choice(_ORDERS, order, "token_order")
    dtype, scaling = _choice(_DTYPES, dtype, "dtype"), _choice(_ROPE_SCALINGS, scaling, "scaling")
    other = 1 if _choice(_DTYPES, out_dtype, "out_dtype") != dtype else 0
    return tuple(_RopeGridParams(batch, heads, kv_heads, n, d, layout, span, len(columns), *four, order, batched, dtype, other,
                                 scaling, orig_len, *real, (ctypes.c_double * ROPE_MAX_AXES)(*step)) for batched in (0, 1))


@dataclass(frozen=True)
class Sizes:
    levels: int
    enrich_levels: int
    n_level: tuple
    topk_level: tuple
    row_offset: tuple
    pyr_rows: int
    n_blocks: int
    keys_per_query: int
    slices: int
    level_idx_offset: tuple
    level_idx_per_slice: int
    scale: float
    coarse_cols: int   # entries per coarse_idx row (levels 1..L)
    enrich_cols: int   # coarse keys per query (columns of levels 1..L_e)


def get_sizes(p: Params) -> Sizes:
    s = _Sizes()
    _check(_load().llsa_get_sizes(ctypes.byref(p.c()), ctypes.byref(s)), "llsa_get_sizes")
    L = s.levels
    return Sizes(L, s.enrich_levels, tuple(s.n_level[:L + 1]), tuple(s.topk_level[:L + 1]),
                 tuple(s.row_offset[:L + 1]), s.pyr_rows, s.n_blocks, s.keys_per_query, s.slices,
                 tuple(s.level_idx_offset[:L + 1]), s.level_idx_per_slice, s.scale, s.coarse_cols, s.enrich_cols)


def workspace_bytes(p: Params, op: int) -> int:
    return int(_load().llsa_workspace_bytes(ctypes.byref(p.c()), op))


def _ptr(t, name, dtype=None):
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    return t.data_ptr()


def _stream(stream):
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _ws(ws):
    if ws is None:
        return None, 0
    return _ptr(ws, "ws"), ws.numel() * ws.element_size()


def _tok_dtype(p: Params):
    return torch.bfloat16 if p.dtype == "bf16" else torch.float32


# ------------------------------------------------------------------ C calls

def llsa_pool(p: Params, q, k, v, pyr, ws=None, stream=None):
    td = _tok_dtype(p)
    w, wb = _ws(ws)
    _check(_load().llsa_pool(ctypes.byref(p.c()), _ptr(q, "q", td), _ptr(k, "k", td), _ptr(v, "v", td),
                             _ptr(pyr, "pyr", torch.float32), w, wb, _stream(stream)), "llsa_pool")


def llsa_select(p: Params, pyr, sel_idx, coarse_idx, level_idx=None, ws=None, stream=None):
    w, wb = _ws(ws)
    _check(_load().llsa_select(ctypes.byref(p.c()), _ptr(pyr, "pyr", torch.float32),
                               _ptr(sel_idx, "sel_idx", torch.int32), _ptr(coarse_idx, "coarse_idx", torch.int32),
                               _ptr(level_idx, "level_idx", torch.int32), w, wb, _stream(stream)), "llsa_select")


def llsa_fwd(p: Params, q, k, v, pyr, sel_idx, coarse_idx, o, lse, ws=None, stream=None):
    td = _tok_dtype(p)
    w, wb = _ws(ws)
    _check(_load().llsa_fwd(ctypes.byref(p.c()), _ptr(q, "q", td), _ptr(k, "k", td), _ptr(v, "v", td),
                            _ptr(pyr, "pyr", torch.float32), _ptr(sel_idx, "sel_idx", torch.int32),
                            _ptr(coarse_idx, "coarse_idx", torch.int32), _ptr(o, "o", td),
                            _ptr(lse, "lse", torch.float32), w, wb, _stream(stream)), "llsa_fwd")


def llsa_index_transpose(p: Params, sel_idx, col_ptr, row_idx, ws, stream=None):
    w, wb = _ws(ws)
    _check(_load().llsa_index_transpose(ctypes.byref(p.c()), _ptr(sel_idx, "sel_idx", torch.int32),
                                        _ptr(col_ptr, "col_ptr", torch.int32), _ptr(row_idx, "row_idx", torch.int32),
                                        w, wb, _stream(stream)), "llsa_index_transpose")


def llsa_select_exhaustive(p: Params, pyr, sel_idx, stream=None):
    """Exhaustive level-1 Top-K: sel_idx int32 [batch*heads, T, min(K, T)]."""
    _check(_load().llsa_select_exhaustive(ctypes.byref(p.c()), _ptr(pyr, "pyr", torch.float32),
                                          _ptr(sel_idx, "sel_idx", torch.int32), _stream(stream)),
           "llsa_select_exhaustive")


def routing_recall(hier_sel, exhaustive_sel) -> float:
    """Share of the exhaustive level-1 Top-K entries that the hierarchical
    selection also holds, over all rows (both int32 [.., T, K] tensors)."""
    h = hier_sel.reshape(-1, hier_sel.shape[-1]).long()
    e = exhaustive_sel.reshape(-1, exhaustive_sel.shape[-1]).long()
    hit = (e[:, :, None] == h[:, None, :]).any(-1)
    return float(hit.double().mean())


def llsa_reorder(p: Params, height: int, width: int, x, out, inverse: bool = False, stream=None):
    """Hierarchical tile order of the N = height * width tokens of x
    [batch, heads, N, d] into out (inverse=True maps back to raster order)."""
    td = _tok_dtype(p)
    _check(_load().llsa_reorder(ctypes.byref(p.c()), int(height), int(width), _ptr(x, "x", td), _ptr(out, "out", td),
                                1 if inverse else 0, _stream(stream)), "llsa_reorder")


def llsa_bwd(p: Params, q, k, v, o, lse, dout, pyr, sel_idx, coarse_idx, col_ptr, row_idx, dq, dk, dv, ws,
             stream=None):
    td = _tok_dtype(p)
    w, wb = _ws(ws)
    i32, f32 = torch.int32, torch.float32
    _check(_load().llsa_bwd(ctypes.byref(p.c()), _ptr(q, "q", td), _ptr(k, "k", td), _ptr(v, "v", td),
                            _ptr(o, "o", td), _ptr(lse, "lse", f32), _ptr(dout, "dout", td), _ptr(pyr, "pyr", f32),
                            _ptr(sel_idx, "sel_idx", i32), _ptr(coarse_idx, "coarse_idx", i32),
                            _ptr(col_ptr, "col_ptr", i32), _ptr(row_idx, "row_idx", i32), _ptr(dq, "dq", td),
                            _ptr(dk, "dk", td), _ptr(dv, "dv", td), w, wb, _stream(stream)), "llsa_bwd")


def _like(t, name, shape, dtype, device):
    """Pointer of a contiguous tensor of exactly this shape and type on device number `device`."""
    if (isinstance(t, torch.Tensor) and t.dtype == dtype and t.shape == shape and t.get_device() == device
            and t.is_contiguous()):
        return t.data_ptr()
    if t is None:
        raise TypeError(f"{name} must be a torch.Tensor")
    ptr = _ptr(t, name, dtype)
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.get_device() != device:
        raise ValueError(f"{name} must be on cuda:{device}, got {t.device}")
    return ptr


def _all_like(tensors, want, device):
    """_like of each tensor and its (name, type, shape) in `want`, in one loop: small calls wait for the host."""
    try:
        for t, (_, dtype, shape) in zip(tensors, want):
            if t.dtype != dtype or t.shape != shape or t.get_device() != device or not t.is_contiguous():
                break
        else:
            return [t.data_ptr() for t in tensors]
    except AttributeError:  # no tensor
        pass
    return [_like(t, name, shape, dtype, device) for t, (name, dtype, shape) in zip(tensors, want)]


_HERE = contextlib.nullcontext()


def _on(t, name):
    """The device of the call: that of its first tensor, which becomes the current one."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    return _HERE if t.get_device() == torch._C._cuda_getDevice() else torch.cuda.device(t.device)


def dense_workspace_bytes(p: DenseParams, op: int) -> int:
    """Workspace of llsa_dense_fwd (OP_DENSE_FWD) or llsa_dense_bwd (OP_DENSE_BWD)."""
    got = p._ws.get(op)
    if got is None:
        got = p._ws[op] = int(_load().llsa_dense_workspace_bytes(p._ref, op))
    return got


def _ws_on(ws, device):
    """The workspace's pointer and bytes, on device number `device`."""
    if ws is not None and isinstance(ws, torch.Tensor) and ws.is_cuda and ws.get_device() != device:
        raise ValueError(f"ws must be on cuda:{device}, got {ws.device}")
    return _ws(ws)


def _lens(p, q_len, k_len, device):
    return tuple(None if x is None else _like(x, name, (p.batch,), torch.int32, device)
                 for x, name in ((q_len, "q_len"), (k_len, "k_len")))


def llsa_dense_fwd(p: DenseParams, q, k, v, o, lse, q_len=None, k_len=None, ws=None, stream=None):
    """Dense attention: o and lse of q over k, v (llsa_dense_fwd of include/llsa.h)."""
    with _on(q, "q"):
        td, dev, (sq, sk, sl) = _tok_dtype(p), q.get_device(), p.shapes()
        ql, kl = (None, None) if q_len is None and k_len is None else _lens(p, q_len, k_len, dev)
        w, wb = _ws_on(ws, dev)
        _check(_load().llsa_dense_fwd(p._ref, _like(q, "q", sq, td, dev), _like(k, "k", sk, td, dev),
                                      _like(v, "v", sk, td, dev), ql, kl, _like(o, "o", sq, td, dev),
                                      _like(lse, "lse", sl, torch.float32, dev), w, wb, _stream(stream)), "llsa_dense_fwd")


def llsa_dense_bwd(p: DenseParams, q, k, v, o, lse, dout, dq, dk, dv, q_len=None, k_len=None, ws=None, stream=None):
    """Gradients of dense attention (llsa_dense_bwd of include/llsa.h)."""
    with _on(q, "q"):
        td, dev, (sq, sk, sl) = _tok_dtype(p), q.get_device(), p.shapes()
        ql, kl = (None, None) if q_len is None and k_len is None else _lens(p, q_len, k_len, dev)
        w, wb = _ws_on(ws, dev)
        _check(_load().llsa_dense_bwd(p._ref, _like(q, "q", sq, td, dev), _like(k, "k", sk, td, dev),
                                      _like(v, "v", sk, td, dev), _like(o, "o", sq, td, dev),
                                      _like(lse, "lse", sl, torch.float32, dev), _like(dout, "dout", sq, td, dev), ql, kl,
                                      _like(dq, "dq", sq, td, dev), _like(dk, "dk", sk, td, dev),
                                      _like(dv, "dv", sk, td, dev), w, wb, _stream(stream)), "llsa_dense_bwd")


def diff_workspace_bytes(p: DiffParams, op: int) -> int:
    """Workspace of llsa_diff_fwd (OP_DIFF_FWD) or llsa_diff_bwd (OP_DIFF_BWD)."""
    got = p._ws.get(op)
    if got is None:
        got = p._ws[op] = int(_load().llsa_diff_workspace_bytes(p._ref, op))
    return got


def llsa_diff_fwd(p: DiffParams, q, k, v, lam, o, o2, lse, q_len=None, k_len=None, ws=None, stream=None):
    """Differential attention: o, o2 (None: not kept) and lse of q over k, v (llsa_diff_fwd of include/llsa.h)."""
    with _on(q, "q"):
        dev = q.get_device()
        q, k, v, lam, o, lse, *kept = _all_like((q, k, v, lam, o, lse) if o2 is None else (q, k, v, lam, o, lse, o2), p._fwd, dev)
        ql, kl = (None, None) if q_len is None and k_len is None else _lens(p, q_len, k_len, dev)
        w, wb = _ws_on(ws, dev)
        _check(_load().llsa_diff_fwd(p._ref, q, k, v, lam, ql, kl, o, kept[0] if kept else None, lse, w, wb, _stream(stream)),
               "llsa_diff_fwd")


def llsa_diff_bwd(p: DiffParams, q, k, v, lam, o, o2, lse, dout, dq, dk, dv, dlam, q_len=None, k_len=None, ws=None, stream=None):
    """Gradients of differential attention (llsa_diff_bwd of include/llsa.h)."""
    with _on(q, "q"):
        dev = q.get_device()
        at = _all_like((q, k, v, lam, o, o2, lse, dout, dq, dk, dv, dlam), p._bwd, dev)
        ql, kl = (None, None) if q_len is None and k_len is None else _lens(p, q_len, k_len, dev)
        w, wb = _ws_on(ws, dev)
        _check(_load().llsa_diff_bwd(p._ref, *at[:8], ql, kl, *at[8:], w, wb, _stream(stream)), "llsa_diff_bwd")


def _strided(t, name, shape, dtype, device):
    """Pointer of a [batch, heads, n, d] tensor whose columns are contiguous, and
    its batch, head and token strides (None: contiguous throughout)."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.get_device() != device:
        raise ValueError(f"{name} must be on cuda:{device}, got {t.device}")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.is_contiguous():
        return t.data_ptr(), None
    s = t.stride()
    if s[3] != 1:
        raise ValueError(f"{name} must have contiguous columns")
    if not any(s[:3]):  # one row for all tokens: zeros mean contiguous to the library
        raise ValueError(f"{name} must not be one row expanded over all tokens")
    return t.data_ptr(), s[:3]


def _rope_strides(views):
    """The C structure of the strides of q, k, q_out, k_out; None where all are contiguous."""
    if not any(views):
        return None
    st = _RopeStrides()
    for field, s in zip((st.q, st.k, st.q_out, st.k_out), views):
        if s is not None:
            field[:] = s
    return ctypes.byref(st)


def llsa_rope(p: RopeParams, q, k, q_out, k_out, pos=None, inverse: bool = False, stream=None):
    """Rotary positions of q and k (None where p.kv_heads is 0) into q_out and
    k_out, in one launch. All may be strided views with contiguous columns, and
    a tensor may be its own output. pos: int32 [n], [n, axes], or either with a
    leading batch dimension. inverse: the negative angles (the gradient)."""
    _rope_call("llsa_rope", p, q, k, q_out, k_out, pos, inverse, stream)


def llsa_rope_grid(p: RopeGridParams, q, k, q_out, k_out, pos=None, inverse: bool = False, stream=None):
    """Rotary positions on up to four axes: llsa_rope's call with the positions,
    columns and frequencies of llsa_rope_grid_params. pos: int32 [n, axes] or
    [batch, n, axes] ([n] or [batch, n] for one axis)."""
    if pos is None and p.extent is None:
        raise ValueError("without an extent positions must be given")
    _rope_call("llsa_rope_grid", p, q, k, q_out, k_out, pos, inverse, stream)


def _rope_call(entry, p, q, k, q_out, k_out, pos, inverse, stream):
    with _on(q, "q"):
        td, dev = _tok_dtype(p), q.get_device()
        to = {"": td, "bf16": torch.bfloat16, "fp32": torch.float32}[getattr(p, "out_dtype", "")]
        shape = (p.batch, p.heads, p.n, p.d)
        a, sa = _strided(q, "q", shape, td, dev)
        c, sc = _strided(q_out, "q_out", shape, to, dev)
        b = d = sb = sd = None
        if p.kv_heads:
            shape = (p.batch, p.kv_heads, p.n, p.d)
            b, sb = _strided(k, "k", shape, td, dev)
            d, sd = _strided(k_out, "k_out", shape, to, dev)
        elif k is not None or k_out is not None:
            raise ValueError("k and k_out must be None where kv_heads is 0")
        at, batched = None, False
        if pos is not None:
            shape = tuple(pos.shape)
            if p.axes == 1 and shape in ((p.n,), (p.batch, p.n)) and shape != (p.n, 1):
                shape += (1,)
            if shape == (p.batch, p.n, p.axes):
                batched = True
            elif shape != (p.n, p.axes):
                raise ValueError(f"pos must have shape [n, axes] or [batch, n, axes], got {tuple(pos.shape)}")
            at = _like(pos, "pos", pos.shape, torch.int32, dev)
        _check(getattr(_load(), entry)(p.c(batched), _rope_strides((sa, sb, sc, sd)), a, b, at, c, d, 1 if inverse else 0,
                                       _stream(stream)), entry)


def llsa_get_status(stream=None) -> int:
    st = ctypes.c_int(0)
    _check(_load().llsa_get_status(_stream(stream), ctypes.byref(st)), "llsa_get_status")
    return st.value


LLSA_TEST_NO_COPIES = 1
LLSA_TEST_FORCE_GROUPED = 2
LLSA_TEST_FORCE_PER_BLOCK = 4
LLSA_TEST_FEW_BLOCKS = 16


def test_set_wait_limit(polls: int = 0, flags: int = 0):
    """Test hook (llsa_test_set_wait_limit): polls before a bounded device wait
    gives up (0: the kernels' own limit) and test switches
    (LLSA_TEST_NO_COPIES: the copy warps issue nothing; LLSA_TEST_FORCE_GROUPED
    / LLSA_TEST_FORCE_PER_BLOCK: which tensor-core forward llsa_fwd takes;
    LLSA_TEST_FEW_BLOCKS: resident dense kernels on three blocks)."""
    _check(_load().llsa_test_set_wait_limit(int(polls), int(flags)), "llsa_test_set_wait_limit")


def llsa_launch_count() -> int:
    return int(_load().llsa_launch_count())


def profile_enable(on: bool = True):
    _load().llsa_profile_enable(1 if on else 0)


def profile_reset():
    _load().llsa_profile_reset()


def profile_only(prefix: str | None = None):
    """Time only kernels whose name starts with `prefix` (None: all)."""
    _load().llsa_profile_only(prefix.encode() if prefix else None)


def profile_read(cap: int = 4096):
    names = (ctypes.c_char_p * cap)()
    ms = (ctypes.c_float * cap)()
    n = _load().llsa_profile_read(names, ms, cap)
    return [(names[i].decode(), float(ms[i])) for i in range(n)]


# ------------------------------------------------------- buffer management

class Buffers:
    """Device buffers of one problem (allocated by torch, owned here)."""

    def __init__(self, p: Params, device="cuda"):
        s = get_sizes(p)
        self.p, self.s = p, s
        bh = s.slices
        dev = torch.device(device)
        td = _tok_dtype(p)
        self.pyr = torch.empty((3, bh, s.pyr_rows, p.d), dtype=torch.float32, device=dev)
        self.sel_idx = torch.empty((bh, s.n_blocks, s.topk_level[1]), dtype=torch.int32, device=dev)
        self.coarse_idx = torch.empty((bh, s.n_blocks, s.coarse_cols), dtype=torch.int32, device=dev)
        self.level_idx = torch.empty((bh, max(1, s.level_idx_per_slice)), dtype=torch.int32, device=dev)
        self.o = torch.empty((p.batch, p.heads, p.n, p.d), dtype=td, device=dev)
        self.lse = torch.empty((p.batch, p.heads, p.n), dtype=torch.float32, device=dev)
        self.col_ptr = torch.empty((bh, s.n_blocks + 1), dtype=torch.int32, device=dev)
        self.row_idx = torch.empty((bh, s.n_blocks * s.topk_level[1]), dtype=torch.int32, device=dev)
        self.ws_f = torch.empty(max(16, workspace_bytes(p, OP_FWD)), dtype=torch.uint8, device=dev)
        self.ws_t = torch.empty(max(16, workspace_bytes(p, OP_TRANSPOSE)), dtype=torch.uint8, device=dev)
        self.ws_b = torch.empty(max(16, workspace_bytes(p, OP_BWD)), dtype=torch.uint8, device=dev)
        # the sparse-index transpose that forward() issues on a side stream
        self._side = None          # that stream (made on first use)
        self._sel_ready = None     # event: the selection it reads is written
        self._transposed = None    # event: col_ptr / row_idx are written
        self._pending = False      # a transpose was issued that backward() has not waited for

    def side_stream(self):
        if self._side is None:
            self._side = torch.cuda.Stream(device=self.sel_idx.device)
            self._sel_ready = torch.cuda.Event()
            self._transposed = torch.cuda.Event()
        return self._side

    def level(self, l: int):
        """I^(l) as [bh, n_l, K_l] (l >= 2) view of level_idx; I^(1) = sel_idx."""
        if l == 1:
            return self.sel_idx
        s = self.s
        off = s.level_idx_offset[l]
        return self.level_idx[:, off:off + s.n_level[l] * s.topk_level[l]].view(-1, s.n_level[l], s.topk_level[l])


def _as_stream(stream, device):
    if stream is None:
        return torch.cuda.current_stream(device)
    if isinstance(stream, torch.cuda.Stream):
        return stream
    return torch.cuda.ExternalStream(int(stream), device=device)


def forward(p: Params, q, k, v, bufs: Buffers | None = None, stream=None) -> Buffers:
    """pool -> select -> fwd. Returns the buffers (o, lse, indices, pyramids).

    The sparse-index transpose that backward() needs depends on the selection
    alone: it is issued here on a side stream, after select, so that it runs
    beside the forward's grouping pass; backward() waits for it."""
    b = bufs or Buffers(p, q.device)
    st = _as_stream(stream, q.device)
    if b._pending:
        st.wait_event(b._transposed)  # the previous transpose still reads sel_idx
    llsa_pool(p, q, k, v, b.pyr, stream=st)
    llsa_select(p, b.pyr, b.sel_idx, b.coarse_idx, b.level_idx, stream=st)
    side = b.side_stream()
    b._sel_ready.record(st)
    side.wait_event(b._sel_ready)
    llsa_index_transpose(p, b.sel_idx, b.col_ptr, b.row_idx, b.ws_t, stream=side)
    b._transposed.record(side)
    b._pending = True
    for t in (b.sel_idx, b.col_ptr, b.row_idx, b.ws_t):
        t.record_stream(side)  # in use there until the transpose is done
    llsa_fwd(p, q, k, v, b.pyr, b.sel_idx, b.coarse_idx, b.o, b.lse, b.ws_f, stream=st)
    return b


def backward(p: Params, q, k, v, dout, b: Buffers, dq=None, dk=None, dv=None, stream=None):
    """bwd after forward() (and its index transpose). Returns (dq, dk, dv)."""
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    st = _as_stream(stream, q.device)
    if b._pending:
        st.wait_event(b._transposed)
        b._pending = False
    else:
        llsa_index_transpose(p, b.sel_idx, b.col_ptr, b.row_idx, b.ws_t, stream=st)
    stream = st
    llsa_bwd(p, q, k, v, b.o, b.lse, dout, b.pyr, b.sel_idx, b.coarse_idx, b.col_ptr, b.row_idx, dq, dk, dv,
             b.ws_b, stream=stream)
    return dq, dk, dv


def _dense_ws(p, op: int, device):
    """The workspace of one call (None where it needs none)."""
    need = (diff_workspace_bytes if isinstance(p, DiffParams) else dense_workspace_bytes)(p, op)
    if need == 0:
        return None
    return torch.empty(need, dtype=torch.uint8, device=device)


def _under(stream, device):
    """What is allocated for a call belongs to the call's stream, whose order then
    keeps it from being used again too early."""
    return _HERE if stream is None else torch.cuda.stream(_as_stream(stream, device))


def dense_forward(p: DenseParams, q, k, v, q_len=None, k_len=None, o=None, lse=None, ws=None, stream=None):
    """Dense attention of q over k, v. Returns (o, lse); what is not given is
    allocated here, on `stream` (None: the current one)."""
    with _under(stream, q.device):
        o = torch.empty_like(q) if o is None else o
        lse = torch.empty(p.shapes()[2], dtype=torch.float32, device=q.device) if lse is None else lse
        ws = _dense_ws(p, OP_DENSE_FWD, q.device) if ws is None else ws
        llsa_dense_fwd(p, q, k, v, o, lse, q_len, k_len, ws, stream)
    return o, lse


def dense_backward(p: DenseParams, q, k, v, o, lse, dout, q_len=None, k_len=None, dq=None, dk=None, dv=None, ws=None,
                   stream=None):
    """Gradients of dense_forward(). Returns (dq, dk, dv)."""
    with _under(stream, q.device):
        dq = torch.empty_like(q) if dq is None else dq
        dk = torch.empty_like(k) if dk is None else dk
        dv = torch.empty_like(v) if dv is None else dv
        ws = _dense_ws(p, OP_DENSE_BWD, q.device) if ws is None else ws
        llsa_dense_bwd(p, q, k, v, o, lse, dout, dq, dk, dv, q_len, k_len, ws, stream)
    return dq, dk, dv


def diff_forward(p: DiffParams, q, k, v, lam, q_len=None, k_len=None, o=None, o2=None, lse=None, ws=None, stream=None,
                 backward: bool = False):
    """Differential attention of q over k, v. Returns (o, lse, o2); what is not given is
    allocated here, on `stream` (None: the current one), o2 only if `backward` says
    that diff_backward() will need it (else it is None)."""
    with _under(stream, q.device):
        so, sl = p.shapes()[3:]
        o = torch.empty(so, dtype=v.dtype, device=q.device) if o is None else o
        o2 = torch.empty(so, dtype=q.dtype, device=q.device) if o2 is None and backward else o2
        lse = torch.empty(sl, dtype=torch.float32, device=q.device) if lse is None else lse
        ws = _dense_ws(p, OP_DIFF_FWD, q.device) if ws is None else ws
        llsa_diff_fwd(p, q, k, v, lam, o, o2, lse, q_len, k_len, ws, stream)
    return o, lse, o2


def diff_backward(p: DiffParams, q, k, v, lam, o, o2, lse, dout, q_len=None, k_len=None, dq=None, dk=None, dv=None, dlam=None,
                  ws=None, stream=None):
    """Gradients of diff_forward(). Returns (dq, dk, dv, dlam)."""
    with _under(stream, q.device):
        dq = torch.empty_like(q) if dq is None else dq
        dk = torch.empty_like(k) if dk is None else dk
        dv = torch.empty_like(v) if dv is None else dv
        dlam = torch.empty_like(lam) if dlam is None else dlam
        ws = _dense_ws(p, OP_DIFF_BWD, q.device) if ws is None else ws
        llsa_diff_bwd(p, q, k, v, lam, o, o2, lse, dout, dq, dk, dv, dlam, q_len, k_len, ws, stream)
    return dq, dk, dv, dlam


def _turn(rope, *args, **kw):
    """llsa_rope or llsa_rope_grid, by the parameters."""
    (llsa_rope_grid if isinstance(rope, RopeGridParams) else llsa_rope)(rope, *args, **kw)


def _check_rope(p, q, k, name="rope"):
    want = (p.batch, p.heads, p.n, p.d)
    if tuple(q.shape) != want or (k is not None and tuple(k.shape) != (p.batch, p.kv_heads, p.n, p.d)):
        raise ValueError(f"{name} is for q {want} and {p.kv_heads} heads of k, got q {tuple(q.shape)}"
                         + ("" if k is None else f" and k {tuple(k.shape)}"))
    for what, t in (("q", q), ("k", k)):
        if t is not None and t.dtype != _tok_dtype(p):
            raise ValueError(f"{what} must be {_tok_dtype(p)}, as {name} says, got {t.dtype}")
    if getattr(p, "out_dtype", "") not in ("", p.dtype):
        raise ValueError(f"{name} must leave q and k their type: out_dtype is for llsa_rope_grid")


def _contiguous(t):
    """t, or a copy where it is not contiguous or does not start on 16 bytes (a view into a flat buffer)."""
    t = t.contiguous()
    return t if t.data_ptr() % 16 == 0 else t.clone(memory_format=torch.contiguous_format)


def _rope_view(t):
    """t, or a contiguous copy where its strides or its first byte are none that llsa_rope takes."""
    if t.is_contiguous():
        return _contiguous(t)
    unit = 16 // t.element_size()
    ok = any(t.stride()[:3]) and t.stride(3) == 1 and t.data_ptr() % 16 == 0 and all(
        t.stride(i) % unit == 0 for i in range(3) if t.shape[i] > 1)
    return t if ok else _contiguous(t)


def _autograd_function():

    class LLSAFunction(torch.autograd.Function):
        """Differentiable LLSA over [batch, heads, N, d] tensors."""

        @staticmethod
        def forward(ctx, q, k, v, block, topk, levels, enrich_levels, scale, token_order, rope, pos):
            ctx.rope = rope
            if rope is None:
                q, k = _contiguous(q), _contiguous(k)
            else:
                q, k = _rotated(rope, q, k, pos)
            v = _contiguous(v)
            p = Params.like(q, block=block, topk=topk, levels=levels, enrich_levels=enrich_levels, scale=scale,
                            token_order=token_order)
            b = forward(p, q, k, v)
            ctx.p, ctx.b = p, b
            ctx.save_for_backward(q, k, v, *([] if rope is None or pos is None else [pos]))
            return b.o

        @staticmethod
        def backward(ctx, do):
            q, k, v, *pos = ctx.saved_tensors
            dq, dk, dv = backward(ctx.p, q, k, v, _contiguous(do), ctx.b)
            if ctx.rope is not None:
                _turn(ctx.rope, dq, dk, dq, dk, pos=pos[0] if pos else None, inverse=True)
            return dq, dk, dv, None, None, None, None, None, None, None, None

    return LLSAFunction


def _rotated(rope, q, k, pos, inverse=False):
    """Head-major contiguous copies of q and k (None allowed) with their positions turned in."""
    _check_rope(rope, q, k)
    q_out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
    k_out = None if k is None else torch.empty(k.shape, dtype=k.dtype, device=k.device)
    _turn(rope, _rope_view(q), None if k is None else _rope_view(k), q_out, k_out, pos=pos, inverse=inverse)
    return q_out, k_out


_FN = None


def llsa_attention(q, k, v, block: int = 16, topk: int = 8, levels: int = 0, enrich_levels: int = -1,
                   scale: float = 0.0, token_order: str = "tile", rope: RopeParams | RopeGridParams | None = None, pos=None):
    """Autograd entry point: o = LLSA(q, k, v). token_order "raster": q, k, v
    (and o, the gradients) are in the raster order of a square image, reordered
    inside the kernels. rope: rotary positions for q and k (with `pos`, or the
    positions that the parameters imply; its token_order is its own); the turned q and k
    are rounded to their type, and so are their gradients before they are turned back."""
    global _FN
    if _FN is None:
        _FN = _autograd_function()
    return _FN.apply(q, k, v, block, topk, levels, enrich_levels, scale, token_order, rope, pos)


# Where dense_attention with rope= keeps bf16 operands in fp32 from the turn to the last
# rounding. Turned q and k rounded to bf16 are the largest error of a step's gradients
# (against 64 bits, 2-norm, 12 heads; in fp32 all are 0.0017): 0.0042 to 0.0044 at 40 columns and
# more whatever the length, 0.0052 to 0.0061 at 8 from 256 to 4,096 tokens, and up to 0.0058
# with four tokens of 64 columns, whose gradients cancel. So those two are always wide.
# Between them it is 0.0047 to 0.0050 at 16 columns and 0.0043 to 0.0047 at 24 and 32, and fp32 takes the
# GPU 5 times as long (12 heads x 4,096 tokens, d = 32 233 us and 1,180): wide where that
# hides behind the call itself, some 300 us of the host (12 heads x 512 tokens 41 us and 107).
_WIDE_TOKENS, _WIDE_ALWAYS, _WIDE_COLUMNS, _WIDE_PAIRS = 16, 8, 32, 1 << 22


def _wide(q, k):
    if q.dtype != torch.bfloat16:
        return False
    d, nk = q.shape[-1], k.shape[-2]
    return (d <= _WIDE_ALWAYS or max(q.shape[-2], nk) <= _WIDE_TOKENS
            or (d <= _WIDE_COLUMNS and q.numel() * nk <= _WIDE_PAIRS * d))  # pairs of a query and a key


# diff_attention with rope= is wide wherever that hides behind the call, whatever the columns: lam's
# gradient is a sum of terms of both signs over all tokens, and with few heads it can come out as
# small as what the rounding of turned q and k makes of it (one to four heads, worst of 24 inputs of
# up to 4,000 tokens: 0.006 to 0.035 off where the other outputs are 0.003; in fp32 0.0036).
# 2^24 pairs of 64 columns take the GPU 350 us. Up to four heads it is wide for four times as many.
_WIDE_DIFF, _FEW_HEADS = (1 << 24) * 64, 4


def _wide_diff(q, k):
    if q.dtype != torch.bfloat16:
        return False
    return _wide(q, k) or q.numel() * k.shape[-2] <= (4 if q.shape[1] <= 2 * _FEW_HEADS else 1) * _WIDE_DIFF


def _check_values(q, v):
    if v.dtype != q.dtype:
        raise ValueError(f"v must be {q.dtype}, got {v.dtype}")


def _positioned(rope, q, k, v, pos, wide=_wide):
    """Contiguous q, k, v with the positions of `rope` (None: none) turned in, and the
    parameters that turn their gradients back."""
    if rope is None:
        q, k = _contiguous(q), _contiguous(k)
    elif wide(q, k):
        _check_rope(rope, q, k)
        _check_values(q, v)
        q, k, v = (t.to(torch.float32, memory_format=torch.contiguous_format) for t in (q, k, v))
        rope = rope.in_fp32()
        _turn(rope, q, k, q, k, pos=pos)
    else:
        q, k = _rotated(rope, q, k, pos)
    return q, k, _contiguous(v), rope


def _dense_functions():
    from torch.autograd.function import once_differentiable

    class DenseFunction(torch.autograd.Function):
        """Differentiable dense attention, with rotary positions if asked."""

        @staticmethod
        def forward(ctx, q, k, v, causal, scale, q_len, k_len, rope, pos):
            ctx.dtype = dtype = q.dtype
            q, k, v, rope = _positioned(rope, q, k, v, pos)
            p = DenseParams.like(q, k, causal=causal, scale=scale)
            o, lse = dense_forward(p, q, k, v, q_len, k_len)
            ctx.p, ctx.rope = p, rope
            ctx.save_for_backward(q, k, v, o, lse, q_len, k_len, pos)
            return o.to(dtype)

        @staticmethod
        @once_differentiable
        def backward(ctx, do):
            q, k, v, o, lse, q_len, k_len, pos = ctx.saved_tensors
            dq, dk, dv = dense_backward(ctx.p, q, k, v, o, lse, _contiguous(do.to(o.dtype)), q_len, k_len)
            if ctx.rope is not None:
                _turn(ctx.rope, dq, dk, dq, dk, pos=pos, inverse=True)
            if dq.dtype != ctx.dtype:
                dq, dk, dv = dq.to(ctx.dtype), dk.to(ctx.dtype), dv.to(ctx.dtype)
            return dq, dk, dv, None, None, None, None, None, None

    class DiffFunction(torch.autograd.Function):
        """Differentiable differential attention, with rotary positions if asked."""

        @staticmethod
        def forward(ctx, q, k, v, lam, causal, scale, q_len, k_len, rope, pos):
            ctx.dtype = q.dtype
            ctx.narrow = grid = None if rope is None or not _wide_diff(q, k) else rope.grid(pos is not None)
            if grid is not None:  # turned into fp32, and the gradients back out of it
                _check_rope(rope, q, k)
                _check_values(q, v)
                x, y = (torch.empty(t.shape, dtype=torch.float32, device=t.device) for t in (q, k))
                llsa_rope_grid(grid.to_fp32(), _rope_view(q), _rope_view(k), x, y, pos=pos)
                q, k, v = x, y, _contiguous(v)
            else:
                q, k, v, rope = _positioned(rope, q, k, v, pos, _wide_diff)
            lam = _contiguous(lam)
            p = DiffParams.like(q, k, lam, causal, scale, v)
            o, lse, o2 = diff_forward(p, q, k, v, lam, q_len, k_len, backward=any(ctx.needs_input_grad))
            ctx.p, ctx.rope = p, rope
            ctx.save_for_backward(q, k, v, lam, o, o2, lse, q_len, k_len, pos)
            return o.to(ctx.dtype)

        @staticmethod
        @once_differentiable
        def backward(ctx, do):
            q, k, v, lam, o, o2, lse, q_len, k_len, pos = ctx.saved_tensors
            dq, dk, dv, dlam = diff_backward(ctx.p, q, k, v, lam, o, o2, lse, _contiguous(do.to(o.dtype)), q_len, k_len)
            if ctx.narrow is not None:
                x, y = (torch.empty(t.shape, dtype=ctx.dtype, device=t.device) for t in (dq, dk))
                llsa_rope_grid(ctx.narrow.from_fp32(), dq, dk, x, y, pos=pos, inverse=True)
                dq, dk = x, y
            elif ctx.rope is not None:
                _turn(ctx.rope, dq, dk, dq, dk, pos=pos, inverse=True)
            if dq.dtype != ctx.dtype:
                dq, dk, dv = dq.to(ctx.dtype), dk.to(ctx.dtype), dv.to(ctx.dtype)
            return dq, dk, dv, dlam, None, None, None, None, None, None

    class RotaryFunction(torch.autograd.Function):
        """Differentiable rotary positions of q and k."""

        @staticmethod
        def forward(ctx, q, k, rope, pos):
            ctx.rope = rope
            ctx.save_for_backward(pos)
            return _rotated(rope, q, k, pos)

        @staticmethod
        @once_differentiable
        def backward(ctx, dq, dk):
            (pos,) = ctx.saved_tensors
            dq, dk = _rotated(ctx.rope, dq, dk, pos, inverse=True)
            return dq, dk, None, None

    return DenseFunction, RotaryFunction, DiffFunction


_DENSE_FNS = None


def _dense_fns():
    global _DENSE_FNS
    if _DENSE_FNS is None:
        _DENSE_FNS = _dense_functions()
    return _DENSE_FNS


def dense_attention(q, k, v, causal: bool = False, scale: float = 0.0, q_len=None, k_len=None,
                    rope: RopeParams | RopeGridParams | None = None, pos=None):
    """Autograd entry point of dense attention: q [batch, heads, nq, d] over k, v
    [batch, kv_heads, nk, d]. q_len, k_len: int32 [batch] valid tokens of a
    padded batch. rope: rotary positions for q and k of the same tokens; the turned
    q and k are rounded to their type before the scores, as rotary() returns them,
    and their gradients before they are turned back. bf16 of up to 8 columns or 16
    tokens stays in fp32 from the turn to the last rounding instead, and so does bf16
    of up to 32 columns and 2^22 pairs of a query and a key. rotary() and
    dense_attention() one after the other round to their type at any size.
    A backward pass that a CUDA graph captures wants leaves made inside the capture
    (x.detach().requires_grad_()), as every autograd function does."""
    return _dense_fns()[0].apply(q, k, v, causal, scale, q_len, k_len, rope, pos)


def diff_attention(q, k, v, lam, causal: bool = False, scale: float = 0.0, q_len=None, k_len=None,
                   rope: RopeParams | RopeGridParams | None = None, pos=None):
    """Autograd entry point of differential attention: o [batch, heads, nq, 2d] =
    (softmax(q1 k1) - lam softmax(q2 k2)) v. q [batch, 2 heads, nq, d] and k [batch,
    2 kv_heads, nk, d] hold the first maps' heads, then the second maps'; v [batch,
    kv_heads, nk, 2d]; lam [heads], bf16 or fp32 whatever the type of the others, or
    a tensor of one element for all heads. q_len, k_len, rope, pos and captured backward passes: as
    dense_attention (rope is for the heads of q and k as they are); with rope, bf16 stays
    in fp32 from the turn to the last rounding where that call's does, and up to 2^30
    products of a pair of a query and a key (both maps' pairs times d), 2^32 with up to four heads. The
    backward pass forms dout . o from o as it was rounded."""
    if not isinstance(lam, torch.Tensor):
        raise TypeError(f"lam must be a torch.Tensor, of one element for all heads or of [heads], not {type(lam).__name__}")
    if lam.numel() == 1:
        lam = lam.reshape(1).expand(q.shape[1] // 2)
    return _dense_fns()[2].apply(q, k, v, lam, causal, scale, q_len, k_len, rope, pos)


def rotary(q, k=None, rope: RopeParams | RopeGridParams | None = None, pos=None):
    """Autograd entry point of rotary positions: (q, k) turned, head-major and
    contiguous (k None: q alone). Strided inputs are read in place."""
    if rope is None:
        rope = RopeParams.like(q, k)
    out = _dense_fns()[1].apply(q, k, rope, pos)
    return out if k is not None else out[0]


def default_scale(d: int) -> float:
    return 1.0 / math.sqrt(d)
