"""Differential attention: what the host refuses, and the sizes it computes, without a
GPU (these calls fail or return before any device work)."""
import copy
import ctypes
import dataclasses
import pickle

import pytest
import torch

import hierarchical_sparse_attention_mean_gb300 as llsa
from hierarchical_sparse_attention_mean_gb300 import build

INVALID, SHAPE, DTYPE, ALIGN, WORKSPACE, UNSUPPORTED = -1, -2, -3, -4, -6, -8
BASE = dict(batch=2, heads=4, nq=100, nk=100, d=64)


@pytest.fixture(scope="module")
def lib():
    build.build()
    return llsa._load()


def fwd(lib, p, ptrs=(16,) * 4, lens=(None, None), outs=(16, None, 16), ws=(None, 0)):
    c = p.c() if isinstance(p, llsa.DiffParams) else p
    return lib.llsa_diff_fwd(ctypes.byref(c), *ptrs, *lens, *outs, *ws, None)


def bwd(lib, p, ptrs=(16,) * 8, lens=(None, None), outs=(16,) * 4, ws=(None, 0)):
    c = p.c() if isinstance(p, llsa.DiffParams) else p
    return lib.llsa_diff_bwd(ctypes.byref(c), *ptrs, *lens, *outs, *ws, None)


@pytest.mark.parametrize("kw,code", [
    (dict(d=60), SHAPE), (dict(d=136), SHAPE), (dict(d=0), SHAPE), (dict(d=-8), SHAPE),
    (dict(heads=6, kv_heads=4), SHAPE), (dict(heads=2, kv_heads=4), SHAPE), (dict(heads=0, kv_heads=2), SHAPE),
    (dict(batch=-1), INVALID), (dict(nq=-1), INVALID), (dict(nk=-1), INVALID), (dict(kv_heads=-1), INVALID), (dict(heads=-1), INVALID),
    (dict(scale=-1.0), INVALID), (dict(scale=float("inf")), INVALID), (dict(scale=float("nan")), INVALID),
    (dict(nq=(1 << 30) + 1), UNSUPPORTED), (dict(nk=(1 << 30) + 1), UNSUPPORTED),
    (dict(heads=(1 << 31) - 1), UNSUPPORTED), (dict(heads=1 << 29, kv_heads=1), UNSUPPORTED),
    (dict(heads=1024, kv_heads=1, nq=1 << 21), UNSUPPORTED),
    (dict(batch=1 << 28, heads=1, nk=1 << 30), UNSUPPORTED), (dict(batch=1 << 20, heads=1 << 10), UNSUPPORTED),
])
def test_parameters_refused(lib, kw, code):
    p = llsa.DiffParams(**{**BASE, **kw})
    assert fwd(lib, p) == code and bwd(lib, p) == code
    assert llsa.diff_workspace_bytes(p, llsa.OP_DIFF_FWD) == 0 and llsa.diff_workspace_bytes(p, llsa.OP_DIFF_BWD) == 0


def test_raw_fields_refused(lib):
    for field, value, code in (("dtype", 2, DTYPE), ("lam_dtype", 2, DTYPE), ("qk_fp32", 2, INVALID), ("causal", 2, INVALID)):
        c = llsa._DiffParams(2, 4, 4, 100, 100, 64, 0, 0, 0, 0, 0.0)
        setattr(c, field, value)
        assert fwd(lib, c) == code and bwd(lib, c) == code
    assert lib.llsa_diff_fwd(None, *([16] * 4), None, None, 16, None, 16, None, 0, None) == INVALID
    assert lib.llsa_diff_workspace_bytes(None, 7) == 0


def test_pointers_refused(lib):
    p = llsa.DiffParams(**BASE)
    for f, count, outs in ((fwd, 4, 3), (bwd, 8, 4)):
        for i in range(count):
            ptrs = [16] * count
            ptrs[i] = None
            assert f(lib, p, ptrs) == INVALID
            ptrs[i] = 24
            assert f(lib, p, ptrs) == ALIGN
        for i in range(outs):
            got = [16] * outs
            got[i] = 8
            assert f(lib, p, outs=got) == ALIGN
            if f is bwd or i != 1:  # o2 need not be kept
                got[i] = None
                assert f(lib, p, outs=got) == INVALID
        assert f(lib, p, lens=(6, None)) == ALIGN and f(lib, p, lens=(None, 2)) == ALIGN


def test_nothing_to_do(lib):
    none = dict(ptrs=(None,) * 4, outs=(None,) * 3)
    assert fwd(lib, llsa.DiffParams(0, 4, 100, 100, 64), **none) == 0
    assert fwd(lib, llsa.DiffParams(2, 0, 100, 100, 64), **none) == 0
    assert fwd(lib, llsa.DiffParams(2, 4, 0, 100, 64), **none) == 0
    assert bwd(lib, llsa.DiffParams(2, 0, 100, 100, 64), ptrs=(None,) * 8, outs=(None,) * 4) == 0
    # no keys: k and v may be NULL, q may not; no tokens: dlam is written all the same
    assert fwd(lib, llsa.DiffParams(2, 4, 10, 0, 64), ptrs=(None,) * 4) == INVALID
    assert bwd(lib, llsa.DiffParams(2, 4, 0, 0, 64), ptrs=(None,) * 8, outs=(None,) * 4) == INVALID


def test_workspace(lib):
    one = llsa.DiffParams(1, 6, 1, 65536, 64)
    for f, op in ((fwd, llsa.OP_DIFF_FWD), (bwd, llsa.OP_DIFF_BWD)):
        need = llsa.diff_workspace_bytes(one, op)
        assert need > 0 and f(lib, one) == WORKSPACE
        assert f(lib, one, ws=(16, need - 1)) == WORKSPACE and f(lib, one, ws=(24, need)) == ALIGN
    assert llsa.diff_workspace_bytes(one, 6) == 0 and llsa.diff_workspace_bytes(one, 9) == 0


def test_binding_refuses(lib):
    for kw in (dict(dtype="fp16"), dict(lam_dtype="fp16"), dict(dtype="fp32", qk_dtype="bf16"), dict(qk_dtype="fp16")):
        with pytest.raises(ValueError):
            llsa.DiffParams(**{**BASE, **kw})
    for value in ((1 << 32) + 100, 1 << 31, -(1 << 31) - 1):
        for field in ("batch", "heads", "kv_heads", "nq", "nk", "d"):
            with pytest.raises(ValueError, match=field):
                llsa.DiffParams(**{**BASE, field: value})
    x = torch.zeros(1, 2, 4, 64)
    with pytest.raises(ValueError, match="two heads"):
        llsa.DiffParams.like(x[:, :1], x)
    with pytest.raises(ValueError, match="two heads"):
        llsa.DiffParams.like(x, torch.zeros(1, 3, 4, 64))
    with pytest.raises(ValueError, match="lam must be"):
        llsa.DiffParams.like(x, x, torch.zeros(1, dtype=torch.float16))
    v, lam = torch.zeros(1, 1, 4, 128), torch.zeros(1)
    with pytest.raises(ValueError, match="CUDA"):
        llsa.diff_attention(x, x, v, lam)
    with pytest.raises(ValueError, match="CUDA"):
        llsa.llsa_diff_fwd(llsa.DiffParams.like(x, x, lam), x, x, v, lam, v, None, torch.zeros(1, 2, 4))


def test_parameters_copy_and_pickle(lib):
    p = llsa.DiffParams(2, 4, 100, 90, 64, kv_heads=2, causal=True, lam_dtype="fp32", scale=0.5, qk_dtype="fp32")
    llsa.diff_workspace_bytes(p, llsa.OP_DIFF_BWD)
    assert p.shapes() == ((2, 8, 100, 64), (2, 4, 90, 64), (2, 2, 90, 128), (2, 4, 100, 128), (2, 8, 100))
    for y in (copy.copy(p), copy.deepcopy(p), pickle.loads(pickle.dumps(p)), dataclasses.replace(p)):
        assert y == p and bytes(y.c()) == bytes(p.c())
    assert dataclasses.replace(p, nq=7).c().nq == 7 and p.c().nq == 100


@pytest.mark.parametrize("b,h,n,d,wide", [
    (1, 6, 64, 64, True), (1, 1, 5792, 64, True), (1, 1, 5793, 64, False), (1, 1, 4096, 128, True), (1, 1, 4097, 128, False),
    (2, 2, 2048, 128, True), (2, 2, 2049, 128, False), (1, 4, 2896, 64, True), (1, 4, 2897, 64, False),
    (1, 8, 1024, 64, True), (1, 8, 1025, 64, False), (2, 5, 1295, 32, True), (2, 5, 1296, 40, False),
    (4, 16, 16, 128, True), (2, 6, 4096, 64, False), (1, 1, 16384, 8, True),
])
def test_where_positions_stay_in_fp32(b, h, n, d, wide):
    q = torch.empty(b, 2 * h, n, d, dtype=torch.bfloat16, device="meta")
    assert llsa._wide_diff(q, q) is wide
    assert llsa._wide_diff(q.float(), q.float()) is False


@pytest.mark.parametrize("n", [60, 4096])  # in fp32 from the turn on, and not
@pytest.mark.parametrize("entry", ["diff", "dense"])
def test_positions_of_another_type_are_refused_at_any_size(entry, n):
    """What the positions say of the types holds whether or not a call keeps bf16 in fp32."""
    heads = 10 if entry == "diff" else 5
    q = torch.zeros(1, heads, n, 64, dtype=torch.bfloat16)
    v = torch.zeros(1, 5, n, 128 if entry == "diff" else 64, dtype=torch.bfloat16)
    if entry == "dense":  # there few columns decide
        q, v = q[..., :24], v[..., :24]
    assert (llsa._wide_diff if entry == "diff" else llsa._wide)(q, q) is (n == 60)

    def call(rope, k=q):
        return llsa.diff_attention(q, k, v, torch.zeros(5), rope=rope) if entry == "diff" else llsa.dense_attention(q, k, v, rope=rope)

    d = q.shape[-1]
    kw = dict(kv_heads=heads, columns=(d - 8, 8), extent=(n // 4, 4))
    grid = llsa.RopeGridParams(1, heads, n, d, **kw)
    line = llsa.RopeParams(1, heads, n, d, kv_heads=heads)
    for rope in (grid, line):
        with pytest.raises(ValueError, match="CUDA"):  # found right up to the device
            call(rope)
        with pytest.raises(ValueError, match="q must be torch.float32"):
            call(dataclasses.replace(rope, dtype="fp32"))
        with pytest.raises(ValueError, match="k must be torch.bfloat16"):
            call(rope, q.float())
    for other in (dataclasses.replace(grid, out_dtype="fp32"), dataclasses.replace(grid, dtype="fp32", out_dtype="bf16")):
        with pytest.raises(ValueError, match="must be torch.float32|out_dtype"):
            call(other)
    call_same = dataclasses.replace(grid, out_dtype="bf16")
    with pytest.raises(ValueError, match="CUDA"):
        call(call_same)


@pytest.mark.parametrize("lam", [0.5, 1, None, [0.5]])
def test_lam_that_is_no_tensor_is_refused_by_name(lam):
    x, v = torch.zeros(1, 2, 4, 64), torch.zeros(1, 1, 4, 128)
    with pytest.raises(TypeError, match="lam must be a torch.Tensor"):
        llsa.diff_attention(x, x, v, lam)
