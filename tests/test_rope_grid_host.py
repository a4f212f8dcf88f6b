"""Rotary positions on several axes: what the host refuses, without a GPU."""
import copy
import ctypes
import dataclasses
import pickle

import pytest
import torch

import hierarchical_sparse_attention_mean_gb300 as llsa
from hierarchical_sparse_attention_mean_gb300 import build

INVALID, SHAPE, DTYPE, ALIGN, UNSUPPORTED = -1, -2, -3, -4, -8
BASE = dict(batch=2, heads=4, n=60, d=64, kv_heads=2, columns=(16, 24, 24), extent=(3, 4, 5))


@pytest.fixture(scope="module")
def lib():
    build.build()
    return llsa._load()


def rope(lib, p, ptrs=(16, 16), pos=None, outs=(32, 32), strides=None, inverse=0):
    c = p.c() if isinstance(p, llsa.RopeGridParams) else p
    return lib.llsa_rope_grid(ctypes.byref(c), strides, *ptrs, pos, *outs, inverse, None)


@pytest.mark.parametrize("kw,code", [
    (dict(d=12), SHAPE), (dict(d=264), SHAPE), (dict(columns=(16, 24, 26)), SHAPE), (dict(columns=(16, 24, 23)), SHAPE),
    (dict(columns=(16, 24, 0)), SHAPE), (dict(columns=(-2, 24, 24)), SHAPE), (dict(columns=(2147483646, 2147483646, 6)), SHAPE),
    (dict(columns=(2, 24, 24), scaling="base", factor=2.0), SHAPE),
    (dict(extent=(3, 4, 6)), SHAPE), (dict(extent=(3, 4, 0)), SHAPE), (dict(extent=None), SHAPE),
    (dict(extent=(65536, 65536, 65536)), SHAPE), (dict(extent=(-3, -4, 5)), INVALID),
    (dict(offset=(2147483646, 0, 0)), INVALID),                                      # positions behind int32
    (dict(token_order="tile"), SHAPE), (dict(token_order="tile", n=75, extent=(3, 5, 5)), SHAPE),
    (dict(token_order="tile", n=32, extent=(1, 2, 16)), SHAPE), (dict(token_order="tile", n=192, extent=(3, 8, 8)), SHAPE),
    (dict(token_order="tile", n=16, columns=(16,), extent=(16,)), INVALID),          # no frame
    (dict(step=(1.0, -1.0, 1.0)), INVALID), (dict(step=(1.0, float("inf"), 1.0)), INVALID), (dict(step=(float("nan"), 1, 1)), INVALID),
    (dict(base=1.0), INVALID), (dict(base=float("nan")), INVALID), (dict(scaling="linear", factor=0.0), INVALID),
    (dict(scaling="wavelength", factor=2.0), INVALID), (dict(scaling="wavelength", factor=2.0, orig_len=10, low=3.0, high=3.0), INVALID),
    (dict(amplitude=float("inf")), INVALID), (dict(amplitude=1e39), INVALID),
    (dict(batch=-1), INVALID), (dict(heads=-1), INVALID), (dict(n=-1), INVALID), (dict(kv_heads=-1), INVALID),
    (dict(heads=(1 << 30) + 1, kv_heads=0), UNSUPPORTED), (dict(batch=1 << 24, heads=1 << 11), UNSUPPORTED),
])
def test_parameters_refused(lib, kw, code):
    assert rope(lib, llsa.RopeGridParams(**{**BASE, **kw})) == code


def test_raw_fields_refused(lib):
    for field, value, code in (("dtype", 2, DTYPE), ("layout", 2, INVALID), ("span", 3, INVALID), ("axes", 0, INVALID), ("axes", 5, INVALID),
                               ("token_order", 2, INVALID), ("pos_batched", 2, INVALID), ("out_other", 2, INVALID), ("scaling", 4, INVALID)):
        c = llsa._RopeGridParams.from_buffer_copy(bytes(llsa.RopeGridParams(**BASE).c()))
        setattr(c, field, value)
        assert rope(lib, c) == code, field
    assert lib.llsa_rope_grid(None, None, 16, 16, None, 32, 32, 0, None) == INVALID


def test_pointers_and_strides_refused(lib):
    p = llsa.RopeGridParams(**BASE)
    assert rope(lib, p, ptrs=(None, 16)) == INVALID and rope(lib, p, ptrs=(16, None)) == INVALID
    assert rope(lib, p, outs=(32, None)) == INVALID and rope(lib, p, outs=(40, 32)) == ALIGN
    assert rope(lib, p, pos=6) == ALIGN and rope(lib, p, inverse=2) == INVALID
    # with positions given, what would imply them is ignored: the call gets as far as the device
    assert rope(lib, llsa.RopeGridParams(**{**BASE, "extent": (7, 7, 7), "token_order": "tile"}), pos=6) == ALIGN
    # into the other type: no tensor is its own output, and strides are in elements of its own type
    up = llsa.RopeGridParams(**{**BASE, "out_dtype": "fp32"})
    assert rope(lib, up, outs=(16, 32)) == INVALID and rope(lib, up, outs=(32, 16)) == INVALID
    st = llsa._RopeStrides()
    st.q_out[:] = [15364, 3840, 64]  # 4 elements more: 16 bytes of fp32, 8 of bf16
    assert rope(lib, p, strides=ctypes.byref(st)) == ALIGN and rope(lib, up, outs=(32, 40), strides=ctypes.byref(st)) == ALIGN
    st = llsa._RopeStrides()
    st.q[:] = [15360, 3840, 60]
    assert rope(lib, p, strides=ctypes.byref(st)) == ALIGN
    st.q[:] = [30720, 64, 512]       # in place, other strides: rows would overwrite rows not yet read
    assert rope(lib, p, ptrs=(16, 16), outs=(16, 32), strides=ctypes.byref(st)) == INVALID
    st = llsa._RopeStrides()
    st.q_out[:] = [15360, 0, 64]     # all heads into one
    assert rope(lib, p, strides=ctypes.byref(st)) == INVALID
    none = dict(ptrs=(None, None), outs=(None, None))
    assert rope(lib, llsa.RopeGridParams(**{**BASE, "batch": 0}), **none) == 0
    assert rope(lib, llsa.RopeGridParams(**{**BASE, "n": 0, "extent": (0, 4, 5)}), **none) == 0


def test_binding_refuses(lib):
    for kw in (dict(columns=()), dict(columns=(8,) * 5), dict(extent=(3, 4)), dict(offset=(1,)), dict(step=(1.0, 1.0)),
               dict(span="both"), dict(layout="pairs"), dict(token_order="z"), dict(dtype="fp16"), dict(out_dtype="fp16"), dict(scaling="ntk")):
        with pytest.raises(ValueError):
            llsa.RopeGridParams(**{**BASE, **kw})
    for value in ((1 << 32) + 2, -(1 << 31) - 1):
        for field in ("batch", "heads", "kv_heads", "n", "d", "orig_len"):
            with pytest.raises(ValueError, match=field):
                llsa.RopeGridParams(**{**BASE, field: value})
        for field in ("columns", "extent", "offset"):
            with pytest.raises(ValueError, match=field):
                llsa.RopeGridParams(**{**BASE, field: (1, value, 1)})
    x = torch.zeros(1, 2, 4, 64)
    p = llsa.RopeGridParams.like(x, columns=(16, 16), extent=(2, 2))
    with pytest.raises(ValueError, match="CUDA"):
        llsa.rotary(x, rope=p)
    with pytest.raises(ValueError, match="positions must be given"):
        llsa.llsa_rope_grid(llsa.RopeGridParams.like(x, columns=(16, 16)), x, None, x, None)
    with pytest.raises(ValueError, match="rope is for"):
        llsa.rotary(x[:, :1], rope=p)


def test_parameters_copy_and_pickle():
    p = llsa.RopeGridParams(**{**BASE, "step": (0.5, 1, 1), "offset": [1, 2, 3]})
    assert p.axes == 3 and p.offset == (1, 2, 3)
    for y in (copy.copy(p), copy.deepcopy(p), pickle.loads(pickle.dumps(p)), dataclasses.replace(p)):
        assert y == p and bytes(y.c()) == bytes(p.c()) and bytes(y.c(True)) == bytes(p.c(True)) and y.c(True).pos_batched == 1
    assert p.in_fp32().dtype == "fp32" and list(p.c().offset) == [1, 2, 3, 0]


@pytest.mark.parametrize("kw,extent", [
    (dict(pos_offset=5), (60,)), (dict(axes=2, width=6), (10, 6)), (dict(axes=2, width=7), None), (dict(axes=2, width=60, rot_dim=32), (1, 60)),
    (dict(rot_dim=20, layout="interleaved", scaling="wavelength", factor=2.0, orig_len=9, low=0.5, amplitude=1.5), (60,)),
])
def test_one_and_two_axes_as_a_grid(lib, kw, extent):
    p = llsa.RopeParams(2, 4, 60, 64, kv_heads=2, **kw)
    g = p.grid()
    if extent is None:
        assert g is None and p.grid(True).extent is None
        return
    assert g is p.grid() and g.extent == extent and g.grid() is g
    assert rope(lib, g, pos=6) == ALIGN and rope(lib, p.grid(True), pos=6) == ALIGN  # checked and found right
    for name in ("layout", "base", "scaling", "factor", "orig_len", "low", "high", "amplitude", "dtype", "batch", "heads", "kv_heads", "n", "d"):
        assert getattr(g, name) == getattr(p, name)
    assert sum(g.columns) == (p.rot_dim or p.d) and g.to_fp32().out_dtype == "fp32" and g.from_fp32().dtype == "fp32"


@pytest.mark.parametrize("kw", [dict(axes=2, width=6, pos_offset=3), dict(width=6), dict(axes=0), dict(axes=3, width=6)])
def test_what_one_and_two_axes_refuse_has_no_grid(lib, kw):
    """Positions that llsa_rope refuses do not become others on their way through a grid."""
    p = llsa.RopeParams(2, 4, 60, 64, kv_heads=2, **kw)
    assert p.grid() is None
    assert lib.llsa_rope(ctypes.byref(p.c()), None, 16, 16, None, 32, 32, 0, None) == INVALID
    given = p.grid(True)  # with positions given, what would imply them is ignored, as in llsa_rope
    code = lib.llsa_rope(ctypes.byref(p.c()), None, 16, 16, 6, 32, 32, 0, None)
    assert (given is None and code == INVALID) if p.axes not in (1, 2) else (given.extent is None and code == ALIGN)
