"""Dense attention and rotary positions: what the host refuses, and the sizes it
computes, without a GPU (these calls fail or return before any device work)."""
import ctypes

import pytest
import torch

import hierarchical_sparse_attention_mean_gb300 as llsa
from hierarchical_sparse_attention_mean_gb300 import build

INVALID, SHAPE, DTYPE, ALIGN, DEVICE, WORKSPACE, UNSUPPORTED = -1, -2, -3, -4, -5, -6, -8


@pytest.fixture(scope="module")
def lib():
    build.build()
    return llsa._load()


def fwd(lib, p, ptrs=(16,) * 3, lens=(None, None), outs=(16, 16), ws=(None, 0)):
    c = p.c() if isinstance(p, llsa.DenseParams) else p
    return lib.llsa_dense_fwd(ctypes.byref(c), *ptrs, *lens, *outs, *ws, None)


def bwd(lib, p, ptrs=(16,) * 6, lens=(None, None), outs=(16,) * 3, ws=(None, 0)):
    return lib.llsa_dense_bwd(ctypes.byref(p.c()), *ptrs, *lens, *outs, *ws, None)


def rope(lib, p, ptrs=(16, 16), pos=None, outs=(32, 32), strides=None, inverse=0):
    return lib.llsa_rope(ctypes.byref(p.c()), strides, *ptrs, pos, *outs, inverse, None)


@pytest.mark.parametrize("kw,code", [
    (dict(d=60), SHAPE), (dict(d=264), SHAPE), (dict(d=0), SHAPE),
    (dict(heads=6, kv_heads=4), SHAPE), (dict(heads=2, kv_heads=4), SHAPE), (dict(heads=0, kv_heads=2), SHAPE),
    (dict(batch=-1), INVALID), (dict(nq=-1), INVALID), (dict(nk=-1), INVALID), (dict(kv_heads=-1), INVALID),
    (dict(scale=-1.0), INVALID), (dict(scale=float("inf")), INVALID), (dict(scale=float("nan")), INVALID),
    (dict(nq=(1 << 30) + 1), UNSUPPORTED), (dict(nk=(1 << 30) + 1), UNSUPPORTED),
    (dict(heads=1024, kv_heads=1, nq=1 << 21), UNSUPPORTED),
    (dict(batch=1 << 20, heads=1 << 10, kv_heads=1 << 10), UNSUPPORTED),
])
def test_dense_parameters_refused(lib, kw, code):
    p = llsa.DenseParams(**{**dict(batch=2, heads=4, nq=100, nk=100, d=64), **kw})
    assert fwd(lib, p) == code and bwd(lib, p) == code
    assert llsa.dense_workspace_bytes(p, llsa.OP_DENSE_FWD) == 0
    assert llsa.dense_workspace_bytes(p, llsa.OP_DENSE_BWD) == 0


def test_dense_raw_fields_refused(lib):
    for field, value, code in (("dtype", 2, DTYPE), ("causal", 2, INVALID)):
        c = llsa._DenseParams(2, 4, 4, 100, 100, 64, 0, 0, 0.0)
        setattr(c, field, value)
        assert fwd(lib, c) == code
    assert lib.llsa_dense_fwd(None, *([16] * 3), None, None, 16, 16, None, 0, None) == INVALID
    assert lib.llsa_dense_workspace_bytes(None, 5) == 0


def test_dense_pointers_refused(lib):
    p = llsa.DenseParams(2, 4, 100, 100, 64)
    for i in range(3):
        ptrs = [16] * 3
        ptrs[i] = None
        assert fwd(lib, p, ptrs) == INVALID
        ptrs[i] = 24
        assert fwd(lib, p, ptrs) == ALIGN
    assert fwd(lib, p, outs=(16, None)) == INVALID and fwd(lib, p, outs=(8, 16)) == ALIGN
    assert fwd(lib, p, lens=(6, None)) == ALIGN
    for i in range(6):
        ptrs = [16] * 6
        ptrs[i] = None
        assert bwd(lib, p, ptrs) == INVALID
    for i in range(3):
        outs = [16] * 3
        outs[i] = 4
        assert bwd(lib, p, outs=outs) == ALIGN


def test_dense_nothing_to_do(lib):
    none = dict(ptrs=(None,) * 3, outs=(None, None))
    assert fwd(lib, llsa.DenseParams(0, 4, 100, 100, 64), **none) == 0
    assert fwd(lib, llsa.DenseParams(2, 0, 100, 100, 64), **none) == 0
    assert fwd(lib, llsa.DenseParams(2, 4, 0, 100, 64), **none) == 0
    assert bwd(lib, llsa.DenseParams(2, 4, 0, 0, 64), ptrs=(None,) * 6, outs=(None,) * 3) == 0
    # no keys: k and v may be NULL, q may not
    assert fwd(lib, llsa.DenseParams(2, 4, 10, 0, 64), ptrs=(None,) * 3) == INVALID


def test_dense_workspace(lib):
    p = llsa.DenseParams(1, 12, 4096, 4096, 64)
    assert llsa.dense_workspace_bytes(p, llsa.OP_DENSE_FWD) == 0   # blocks enough: no split
    # the backward keeps two numbers per query row
    assert llsa.dense_workspace_bytes(p, llsa.OP_DENSE_BWD) == 2 * 12 * 4096 * 4
    one = llsa.DenseParams(1, 12, 1, 65536, 64)
    assert llsa.dense_workspace_bytes(one, llsa.OP_DENSE_FWD) > 0
    assert fwd(lib, one) == WORKSPACE and bwd(lib, p) == WORKSPACE
    need = llsa.dense_workspace_bytes(one, llsa.OP_DENSE_FWD)
    assert fwd(lib, one, ws=(16, need - 1)) == WORKSPACE and fwd(lib, one, ws=(24, need)) == ALIGN
    assert llsa.dense_workspace_bytes(one, 4) == 0 and llsa.dense_workspace_bytes(one, 7) == 0


@pytest.mark.parametrize("kw,code", [
    (dict(d=12), SHAPE), (dict(d=264), SHAPE), (dict(rot_dim=65), SHAPE), (dict(rot_dim=66), SHAPE), (dict(rot_dim=-2), SHAPE),
    (dict(rot_dim=62, axes=2, width=4), SHAPE), (dict(rot_dim=2, scaling="base", factor=2.0), SHAPE),
    (dict(axes=3), INVALID), (dict(axes=0), INVALID), (dict(axes=2), INVALID),      # no width, no positions
    (dict(axes=2, width=-4), INVALID), (dict(width=4), INVALID),                     # a width that nothing reads
    (dict(axes=2, width=8, pos_offset=1), INVALID),
    (dict(axes=2, width=8, token_order="tile"), SHAPE),                              # 100 tokens are no 8 x 8 image
    (dict(axes=2, width=10, token_order="tile"), SHAPE),                             # nor is 10 a power of 4
    (dict(base=1.0), INVALID), (dict(base=float("nan")), INVALID), (dict(base=float("inf")), INVALID),
    (dict(scaling="linear", factor=0.0), INVALID), (dict(scaling="linear", factor=float("nan")), INVALID),
    (dict(scaling="wavelength", factor=2.0), INVALID),                               # no orig_len
    (dict(scaling="wavelength", factor=2.0, orig_len=10, low=3.0, high=3.0), INVALID),
    (dict(amplitude=float("inf")), INVALID), (dict(amplitude=float("nan")), INVALID),
    (dict(batch=-1), INVALID), (dict(heads=-1), INVALID), (dict(n=-1), INVALID), (dict(kv_heads=-1), INVALID),
    (dict(pos_offset=2147483647), INVALID),                                          # positions behind int32
])
def test_rope_parameters_refused(lib, kw, code):
    p = llsa.RopeParams(**{**dict(batch=2, heads=4, n=100, d=64, kv_heads=2), **kw})
    assert rope(lib, p) == code


def test_rope_pointers_and_strides_refused(lib):
    p = llsa.RopeParams(2, 4, 100, 64, kv_heads=2)
    assert rope(lib, p, ptrs=(None, 16)) == INVALID and rope(lib, p, ptrs=(16, None)) == INVALID
    assert rope(lib, p, outs=(32, None)) == INVALID and rope(lib, p, outs=(40, 32)) == ALIGN
    assert rope(lib, p, pos=6) == ALIGN
    assert rope(lib, p, inverse=2) == INVALID
    # with positions given, what would imply them is ignored: the call gets as far as the device
    given = llsa.RopeParams(2, 4, 100, 64, kv_heads=2, width=7, pos_offset=2147483647)
    assert rope(lib, given, pos=6) == ALIGN
    st = llsa._RopeStrides()
    st.q[:] = [25600, 6400, 60]      # a token every 120 bytes
    assert rope(lib, p, strides=ctypes.byref(st)) == ALIGN
    st.q[:] = [51200, 64, 512]       # in place, other strides: rows would overwrite rows not yet read
    assert rope(lib, p, ptrs=(16, 16), outs=(16, 32), strides=ctypes.byref(st)) == INVALID
    st = llsa._RopeStrides()
    st.q_out[:] = [25600, 0, 64]     # all heads into one
    assert rope(lib, p, strides=ctypes.byref(st)) == INVALID
    assert rope(lib, llsa.RopeParams(0, 4, 100, 64), (None, None), outs=(None, None)) == 0
    assert rope(lib, llsa.RopeParams(2, 4, 0, 64), (None, None), outs=(None, None)) == 0
    assert lib.llsa_rope(None, None, 16, 16, None, 32, 32, 0, None) == INVALID


def test_names_refused():
    with pytest.raises(ValueError):
        llsa.DenseParams(1, 1, 1, 1, 64, dtype="fp16")
    for kw in (dict(layout="pairs"), dict(scaling="ntk"), dict(token_order="z"), dict(dtype="fp16")):
        with pytest.raises(ValueError):
            llsa.RopeParams(1, 1, 1, 64, **kw)
    with pytest.raises(ValueError):
        llsa.DenseParams.like(torch.zeros(1, 1, 4, 8, dtype=torch.float16), torch.zeros(1, 1, 4, 8))


def test_binding_refuses_host_tensors(lib):
    x = torch.zeros(1, 2, 4, 64)
    p = llsa.DenseParams.like(x, x)
    with pytest.raises(ValueError, match="CUDA"):
        llsa.llsa_dense_fwd(p, x, x, x, x, torch.zeros(1, 2, 4))
    with pytest.raises(ValueError, match="CUDA"):
        llsa.dense_attention(x, x, x)
    with pytest.raises(ValueError, match="CUDA"):
        llsa.rotary(x, x)
    with pytest.raises(TypeError):
        llsa.llsa_rope(llsa.RopeParams.like(x), None, None, x, None)


def test_parameters_copy_and_pickle(lib):
    import copy
    import dataclasses
    import pickle
    p = llsa.DenseParams(2, 4, 100, 90, 64, kv_heads=2, causal=True, scale=0.5)
    r = llsa.RopeParams(2, 4, 256, 64, kv_heads=2, axes=2, width=16, token_order="tile")
    r.c(), r.c(True), llsa.dense_workspace_bytes(p, llsa.OP_DENSE_BWD)
    for x in (p, r):
        for y in (copy.copy(x), copy.deepcopy(x), pickle.loads(pickle.dumps(x)), dataclasses.replace(x)):
            assert y == x and bytes(y.c()) == bytes(x.c())
    assert dataclasses.replace(p, nq=7).c().nq == 7 and p.c().nq == 100


@pytest.mark.parametrize("kw", [dict(heads=(1 << 31) - 1, kv_heads=(1 << 31) - 1), dict(batch=(1 << 31) - 1, n=(1 << 31) - 1),
                                dict(batch=1 << 20, n=1 << 15)])
def test_rope_sizes_refused(lib, kw):
    p = llsa.RopeParams(**{**dict(batch=2, heads=4, n=100, d=64, kv_heads=2), **kw})
    assert rope(lib, p) == UNSUPPORTED


@pytest.mark.parametrize("kw", [
    dict(batch=1 << 28, heads=1, nk=1 << 30),                # 2^64 elements of k
    dict(batch=1 << 30, heads=1, nk=1 << 30, d=16),          # again
    dict(batch=1 << 28, heads=1, nq=1 << 30),                # of q
    dict(batch=1 << 29, heads=1, nk=1 << 29, d=256),
    dict(batch=3 << 20, heads=10, nk=(1 << 30) - 5, d=248),
])
def test_dense_sizes_behind_64_bits_refused(lib, kw):
    p = llsa.DenseParams(**{**dict(batch=2, heads=4, nq=100, nk=100, d=64), **kw})
    assert fwd(lib, p) == UNSUPPORTED and bwd(lib, p) == UNSUPPORTED
    assert llsa.dense_workspace_bytes(p, llsa.OP_DENSE_FWD) == 0
    assert llsa.dense_workspace_bytes(p, llsa.OP_DENSE_BWD) == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_tensors_off_16_bytes_are_copied(dtype):
    """A contiguous view that starts inside a vector is no input of the kernels: a copy is."""
    flat = torch.arange(1 + 2 * 3 * 5 * 8, dtype=dtype)
    for take in (llsa._contiguous, llsa._rope_view):
        view = flat[1:].view(2, 3, 5, 8)
        assert view.is_contiguous() and view.data_ptr() % 16 != 0
        got = take(view)
        assert got.data_ptr() % 16 == 0 and got.is_contiguous() and torch.equal(got, view)
        whole = flat[:-1].view(2, 3, 5, 8)
        assert take(whole) is whole
        turned = take(flat[1:].view(2, 5, 3, 8).transpose(1, 2))
        assert turned.data_ptr() % 16 == 0 and torch.equal(turned, flat[1:].view(2, 5, 3, 8).transpose(1, 2))


@pytest.mark.parametrize("b,h,n,d,wide", [
    (1, 12, 16, 64, True), (1, 12, 17, 64, False), (64, 16, 16, 128, True),    # a handful of tokens
    (1, 12, 16384, 8, True),                                                    # a handful of columns
    (1, 12, 512, 32, True), (1, 12, 600, 32, False), (48, 12, 256, 16, False),  # up to what hides behind the call
    (1, 12, 16384, 32, False), (1, 4, 1024, 32, True), (1, 4, 1025, 24, False), (1, 1, 100, 40, False),
])
def test_where_rotary_attention_stays_in_fp32(b, h, n, d, wide):
    q = torch.empty(b, h, n, d, dtype=torch.bfloat16, device="meta")
    assert llsa._wide(q, q) is wide
    assert llsa._wide(q.float(), q.float()) is False


@pytest.mark.parametrize("heads,kv", [((1 << 31) - 1, (1 << 31) - 1), ((1 << 30) + 1, 0), (1 << 30, 1)])
def test_rope_heads_refused(lib, heads, kv):
    """Few elements, but more heads than a launch counts."""
    p = llsa.RopeParams(1, heads, 1, 8, kv_heads=kv)
    assert rope(lib, p) == UNSUPPORTED


@pytest.mark.parametrize("amplitude", [1e39, -1e300])
def test_rope_amplitudes_refused(lib, amplitude):
    """Finite, but not in the kernel's fp32."""
    assert rope(lib, llsa.RopeParams(2, 4, 100, 64, kv_heads=2, amplitude=amplitude)) == INVALID
    assert rope(lib, llsa.RopeParams(2, 4, 100, 64, kv_heads=2, amplitude=amplitude * 1e-30 if amplitude > 0 else -1e38), pos=6) == ALIGN


WRAPS = [(1 << 32) + 100, 1 << 31, -(1 << 31) - 1, (1 << 32) + 2]


@pytest.mark.parametrize("value", WRAPS)
def test_parameters_behind_32_bits_refused(value):
    """Not cut to their low bits: 2^32 + 100 tokens are not 100, position 2^32 + 2 is not 2."""
    for field in ("batch", "heads", "kv_heads", "nq", "nk", "d"):
        with pytest.raises(ValueError, match=field):
            llsa.DenseParams(**{**dict(batch=2, heads=4, nq=100, nk=100, d=64), field: value})
    for field in ("batch", "heads", "kv_heads", "n", "d", "rot_dim", "axes", "width", "pos_offset", "orig_len"):
        with pytest.raises(ValueError, match=field):
            llsa.RopeParams(**{**dict(batch=2, heads=4, n=100, d=64), field: value})
    q = torch.empty(1, 1, abs(value), 8, dtype=torch.bfloat16, device="meta")
    with pytest.raises(ValueError, match="32 bits"):
        llsa.DenseParams.like(q, q)
    with pytest.raises(ValueError, match="32 bits"):
        llsa.RopeParams.like(q)


def test_a_workspace_on_another_device_is_refused():
    class Far(torch.Tensor):  # stands for a tensor on a second GPU
        is_cuda = property(lambda self: True)

        def get_device(self):
            return 1

    ws = torch.zeros(64, dtype=torch.uint8).as_subclass(Far)
    assert llsa._ws_on(ws, 1) == (ws.data_ptr(), 64) and llsa._ws_on(None, 0) == (None, 0)
    with pytest.raises(ValueError, match="ws must be on cuda:0"):
        llsa._ws_on(ws, 0)
    with pytest.raises(TypeError):
        llsa._ws_on(64, 0)
