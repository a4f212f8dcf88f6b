"""Rotary positions on the GPU against their formulas in 64 bits."""
import pytest
import torch

import hierarchical_sparse_attention_mean_gb300 as llsa
from hierarchical_sparse_attention_mean_gb300 import build

import dense_ref as ref

pytestmark = pytest.mark.gpu
T = {"bf16": torch.bfloat16, "fp32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()


def rand(shape, dtype, seed):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(T[dtype])


def digits(t, side):
    """(row, column) of tile positions t: base-16 digits, each a row and a column digit in base 4."""
    r, c, place = torch.zeros_like(t), torch.zeros_like(t), 1
    while place < side:
        r, c = r + place * ((t & 15) >> 2), c + place * (t & 3)
        t, place = t >> 4, place * 4
    return torch.stack([r, c], -1)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("inverse", [False, True])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("d,rot,axes", [(64, 0, 1), (64, 0, 2), (128, 64, 1), (8, 0, 1), (8, 4, 2), (40, 20, 1), (40, 12, 2),
                                        (72, 0, 1), (256, 0, 2), (16, 6, 1), (16, 2, 1)])
def test_layouts_and_parts_of_the_head(d, rot, axes, layout, inverse, dtype):
    b, h, kv, n = 2, 3, 2, 37
    q, k = rand((b, h, n, d), dtype, d), rand((b, kv, n, d), dtype, d + 1)
    pos = torch.randint(-5000, 5000, (b, n, axes), generator=torch.Generator().manual_seed(3), dtype=torch.int32)
    qc, kc = q.cuda(), k.cuda()
    p = llsa.RopeParams.like(qc, kc, rot_dim=rot, layout=layout, axes=axes)
    qo, ko = torch.full_like(qc, 9.0), torch.full_like(kc, 9.0)
    llsa.llsa_rope(p, qc, kc, qo, ko, pos=pos.cuda(), inverse=inverse)
    torch.cuda.synchronize()
    for x, got in ((q, qo), (k, ko)):
        want = ref.rotary(x, pos, rot=rot, layout=layout, axes=axes, inverse=inverse, dtype=T[dtype])
        ref.check("out", got, want)
        assert torch.equal(got.cpu()[..., (rot or d):], x[..., (rot or d):])   # the rest is a copy
    # in place
    llsa.llsa_rope(p, qc, kc, qc, kc, pos=pos.cuda(), inverse=inverse)
    assert torch.equal(qc, qo) and torch.equal(kc, ko)


@pytest.mark.parametrize("scaling,kw", [("none", {}), ("linear", {"factor": 8.0}), ("base", {"factor": 4.0}),
                                        ("wavelength", {"factor": 8.0, "orig_len": 4096}),
                                        ("wavelength", {"factor": 2.5, "orig_len": 64, "low": 0.5, "high": 4.0}),
                                        ("linear", {"factor": 0.05})])
def test_scalings(scaling, kw):
    x = rand((1, 2, 50, 64), "fp32", 1)
    xc = x.cuda()
    pos = (torch.arange(50, dtype=torch.int32) * 1999)[:, None]
    p = llsa.RopeParams.like(xc, scaling=scaling, **kw)
    out = torch.empty_like(xc)
    llsa.llsa_rope(p, xc, None, out, None, pos=pos.cuda())
    ref.check("out", out, ref.rotary(x, pos[None], scaling=scaling, dtype=torch.float32, **kw))
    # an amplitude of the caller's
    llsa.llsa_rope(llsa.RopeParams.like(xc, scaling=scaling, amplitude=0.75, **kw), xc, None, out, None, pos=pos.cuda())
    ref.check("out", out, ref.rotary(x, pos[None], scaling=scaling, amplitude=0.75, dtype=torch.float32, **kw))


def test_far_positions_keep_their_angles():
    x = rand((1, 1, 6, 64), "fp32", 2)
    pos = torch.tensor([0, 1, 16777217, 2147483647, -2147483648, -3], dtype=torch.int32)[:, None]
    xc, out = x.cuda(), torch.empty(1, 1, 6, 64, device="cuda")
    llsa.llsa_rope(llsa.RopeParams.like(xc), xc, None, out, None, pos=pos.cuda())
    ref.check("out", out, ref.rotary(x, pos[None].long(), dtype=torch.float32))


@pytest.mark.parametrize("shape", ["n", "n,axes", "b,n", "b,n,axes"])
def test_position_shapes(shape):
    b, n = 2, 9
    x = rand((b, 1, n, 32), "fp32", 4).cuda()
    base = torch.randint(0, 999, (b, n), generator=torch.Generator().manual_seed(5), dtype=torch.int32)
    pos = {"n": base[0], "n,axes": base[0][:, None], "b,n": base, "b,n,axes": base[..., None]}[shape].contiguous()
    full = (base if shape.startswith("b") else base[:1].expand(b, n))[..., None]
    out = torch.empty_like(x)
    llsa.llsa_rope(llsa.RopeParams.like(x), x, None, out, None, pos=pos.cuda())
    ref.check("out", out, ref.rotary(x.cpu(), full, dtype=torch.float32))


@pytest.mark.parametrize("order,width,n", [("raster", 7, 45), ("raster", 1, 5), ("tile", 16, 256), ("tile", 4, 16), ("tile", 64, 4096)])
def test_implied_image_positions(order, width, n):
    x = rand((1, 2, n, 32), "bf16", 6)
    xc = x.cuda()
    t = torch.arange(n)
    pos = torch.stack([t // width, t % width], -1) if order == "raster" else digits(t, width)
    out = torch.empty_like(xc)
    llsa.llsa_rope(llsa.RopeParams.like(xc, axes=2, width=width, token_order=order), xc, None, out, None)
    ref.check("out", out, ref.rotary(x, pos[None], axes=2, dtype=torch.bfloat16))


def test_tile_order_agrees_with_the_reordering():
    """Turning in tile order is turning in raster order, then llsa_reorder."""
    n, side = 4096, 64
    x = rand((1, 2, n, 64), "bf16", 8).cuda()
    a, b, c, d = (torch.empty_like(x) for _ in range(4))
    llsa.llsa_rope(llsa.RopeParams.like(x, axes=2, width=side), x, None, a, None)
    p = llsa.Params(1, 2, n, 64)
    llsa.llsa_reorder(p, side, side, a, b)
    llsa.llsa_reorder(p, side, side, x, c)
    llsa.llsa_rope(llsa.RopeParams.like(x, axes=2, width=side, token_order="tile"), c, None, d, None)
    assert torch.equal(b, d)


@pytest.mark.parametrize("n,offset", [(1, 777777), (3, -2), (1000, 100000)])
def test_offset_and_small_calls(n, offset):
    q, k = rand((3, 5, n, 64), "bf16", n), rand((3, 1, n, 64), "bf16", n + 1)
    qc, kc = q.cuda(), k.cuda()
    p = llsa.RopeParams.like(qc, kc, pos_offset=offset)
    pos = (torch.arange(n) + offset)[None, :, None]
    qo, ko = llsa.rotary(qc, kc, p)
    ref.check("q", qo, ref.rotary(q, pos, dtype=torch.bfloat16))
    ref.check("k", ko, ref.rotary(k, pos, dtype=torch.bfloat16))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_packed_projection_in_and_out(dtype):
    """Views of a [batch, n, heads, d] projection, both ways, the neighbours untouched."""
    b, n, h, kv, d = 2, 33, 4, 2, 64
    w = rand((b, n, h + 2 * kv, d), dtype, 10)
    wc = w.cuda()
    v = wc.permute(0, 2, 1, 3)
    q, k = v[:, :h], v[:, h:h + kv]
    p = llsa.RopeParams.like(q, k)
    qo, ko = llsa.rotary(q, k, p)
    pos = torch.arange(n)[None, :, None]
    u = T[dtype]
    ref.check("q", qo, ref.rotary(w.permute(0, 2, 1, 3)[:, :h], pos, dtype=u))
    ref.check("k", ko, ref.rotary(w.permute(0, 2, 1, 3)[:, h:h + kv], pos, dtype=u))
    back = torch.full_like(wc, 5.0)
    bv = back.permute(0, 2, 1, 3)
    llsa.llsa_rope(p, qo, ko, bv[:, :h], bv[:, h:h + kv], inverse=True)
    ref.check("back", bv[:, :h], ref.rotary(qo.cpu(), pos, inverse=True, dtype=u))
    assert bool((bv[:, h + kv:] == 5.0).all())


def test_broadcast_inputs():
    """Rows shared by heads or batch entries are read in place; one row for all is copied first."""
    x = rand((2, 1, 19, 64), "fp32", 21)
    pos = torch.arange(19)[None, :, None]
    q = x.cuda().expand(2, 3, 19, 64)
    p = llsa.RopeParams.like(q)
    ref.check("q", llsa.rotary(q, rope=p), ref.rotary(x.expand(2, 3, 19, 64), pos, dtype=torch.float32))
    row = rand((64,), "fp32", 22)
    one = row.cuda().expand(2, 3, 19, 64)
    ref.check("one", llsa.rotary(one, rope=p), ref.rotary(row.expand(2, 3, 19, 64), pos, dtype=torch.float32))
    with pytest.raises(ValueError, match="expanded"):
        llsa.llsa_rope(p, one, None, torch.empty(2, 3, 19, 64, device="cuda"), None)


def test_columns_behind_the_turned_ones_may_hold_anything():
    x = rand((1, 1, 8, 16), "bf16", 11)
    x[..., 6:] = float("inf")
    x[0, 0, 3, 9] = float("nan")
    for layout in ("half", "interleaved"):
        xc = x.cuda()
        out = torch.empty_like(xc)
        llsa.llsa_rope(llsa.RopeParams.like(xc, rot_dim=6, layout=layout), xc, None, out, None)
        assert bool(torch.isfinite(out[..., :6]).all())
        assert torch.equal(out.cpu()[..., 6:].view(torch.int16), x[..., 6:].view(torch.int16))


def test_autograd_is_the_inverse_turn():
    q, k = (rand((2, h, 21, 64), "fp32", 12 + h).cuda().requires_grad_() for h in (4, 2))
    p = llsa.RopeParams.like(q, k, axes=2, width=7, scaling="wavelength", factor=4.0, orig_len=16)
    outs = llsa.rotary(q, k, p)
    g = [torch.randn_like(t) for t in outs]
    got = torch.autograd.grad(outs, (q, k), g)
    want = [torch.empty_like(t) for t in g]
    llsa.llsa_rope(p, *g, *want, inverse=True)
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    # <R x, g> = <x, R^T g>
    outs = [o.detach() for o in outs]
    lhs = sum((o.double() * t.double()).sum() for o, t in zip(outs, g))
    rhs = sum((x.double() * t.double()).sum() for x, t in zip((q.detach(), k.detach()), got))
    size = sum((o.double().abs() * t.double().abs()).sum() for o, t in zip(outs, g))
    assert abs(float(lhs - rhs)) <= 2.0 ** -20 * float(size)
    # q alone
    (only,) = torch.autograd.grad(llsa.rotary(q, rope=llsa.RopeParams.like(q)).sum(), (q,))
    assert only.shape == q.shape


def test_captured_graph():
    x = rand((1, 4, 100, 64), "bf16", 20).cuda()
    p = llsa.RopeParams.like(x, x)
    a, b = torch.empty_like(x), torch.empty_like(x)
    llsa.llsa_rope(p, x, x, a, b)
    graph = torch.cuda.CUDAGraph()
    c, d = torch.zeros_like(x), torch.zeros_like(x)
    with torch.cuda.graph(graph):
        llsa.llsa_rope(p, x, x, c, d)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(a, c) and torch.equal(b, d)


def test_one_token_positions():
    """[n, axes] with one token serves every entry; [batch, n] gives each its own."""
    q = rand((3, 2, 1, 64), "fp32", 30)
    qc = q.cuda()
    p = llsa.RopeParams.like(qc)
    for pos, full in (([[7]], [[[7]]]), ([7], [[[7]]]), ([[7], [8], [-9]], [[[7]], [[8]], [[-9]]])):
        out = torch.empty_like(qc)
        llsa.llsa_rope(p, qc, None, out, None, pos=torch.tensor(pos, dtype=torch.int32, device="cuda"))
        ref.check("out", out, ref.rotary(q, torch.tensor(full), dtype=torch.float32))


PI = "3.14159265358979323846264338327950288419716939937510582097494459230781640628620899862803"


def turns_per_position(seg, i, base=10000.0, scaling="none", factor=1.0, orig_len=0, low=1.0, high=32.0):
    """A pair's frequency in turns, to 60 digits."""
    from decimal import Decimal, localcontext
    with localcontext() as c:
        c.prec = 60
        b, f, two_pi = Decimal(base), Decimal(factor), 2 * Decimal(PI)
        if scaling == "base":
            b *= f ** (Decimal(seg) / (seg - 2))
        w = b ** (Decimal(-2 * i) / seg)
        if scaling == "linear":
            w /= f
        if scaling == "wavelength":
            g = min(Decimal(1), max(Decimal(0), (orig_len * w / two_pi - Decimal(low)) / (Decimal(high) - Decimal(low))))
            w *= g + (1 - g) / f
        return w / two_pi


@pytest.mark.parametrize("d,kw", [(64, {}), (128, {"base": 500000.0}), (64, {"scaling": "linear", "factor": 8.0}),
                                  (64, {"scaling": "linear", "factor": 0.05}), (72, {"scaling": "base", "factor": 16.0}),
                                  (64, {"scaling": "wavelength", "factor": 8.0, "orig_len": 4096, "amplitude": 1.0})])
def test_angles_are_as_good_as_stated(d, kw):
    """Unit vectors, so that the outputs are cosine and sine: off by the stated error of the
    angle and by 2 ulp of sincospif."""
    import math
    from decimal import Decimal, localcontext
    at = [0, 1, -1, 2, 3, 37, 1000, 4095, -99999, 777777, 1 << 24, (1 << 24) + 1, 123456789, -(1 << 30), (1 << 31) - 1, -(1 << 31)]
    x = torch.zeros(1, 1, len(at), d)
    x[..., :d // 2] = 1.0
    out = torch.empty_like(x, device="cuda")
    p = llsa.RopeParams(1, 1, len(at), d, dtype="fp32", **kw)
    llsa.llsa_rope(p, x.cuda(), None, out, None, pos=torch.tensor(at, dtype=torch.int32, device="cuda"))
    got = out.cpu().double()[0, 0]
    kw = {k: v for k, v in kw.items() if k != "amplitude"}
    for i in range(d // 2):
        f = turns_per_position(d, i, **kw)
        for t, pos in enumerate(at):
            with localcontext() as c:
                c.prec = 60
                turn = f * pos
                turn = float(turn - turn.to_integral_value())
            far = 2.0 ** -26 + 2.0 ** -32 + abs(pos) * max(1.0, 2 * math.pi * float(f)) * 2.0 ** -54
            for value, want in ((got[t, i], math.cos(2 * math.pi * turn)), (got[t, i + d // 2], math.sin(2 * math.pi * turn))):
                assert abs(float(value) - want) <= 2 * math.pi * far + 2.0 ** -23 * abs(want) + 2.0 ** -40, (i, pos)


@pytest.mark.parametrize("h,kv,n", [(65536, 0, 1), (65535, 1, 1), (50000, 90000, 3), (131072, 3, 1)])
def test_many_heads(h, kv, n):
    """More heads than a grid has blocks in its second dimension."""
    q, k = rand((1, h, n, 8), "fp32", 40), rand((1, kv, n, 8), "fp32", 41)
    qc, kc = q.cuda(), k.cuda() if kv else None
    p = llsa.RopeParams.like(qc, kc, pos_offset=5)
    pos = (torch.arange(n) + 5)[None, :, None]
    out = llsa.rotary(qc, kc, p)
    ref.check("q", out[0] if kv else out, ref.rotary(q, pos, dtype=torch.float32))
    if kv:
        ref.check("k", out[1], ref.rotary(k, pos, dtype=torch.float32))


@pytest.mark.parametrize("factor", [1.0, 0.5, 1e-5])
def test_wavelength_scaling_that_stretches_nothing_keeps_lengths(factor):
    """The amplitude follows the logarithm of the factor above 1 alone."""
    x = rand((1, 2, 50, 64), "fp32", 50)
    xc, out = x.cuda(), torch.empty(1, 2, 50, 64, device="cuda")
    pos = (torch.arange(50, dtype=torch.int32) * 7)[:, None]
    kw = dict(scaling="wavelength", factor=factor, orig_len=64)
    llsa.llsa_rope(llsa.RopeParams.like(xc, **kw), xc, None, out, None, pos=pos.cuda())
    value, bound = ref.rotary(x, pos[None], amplitude=1.0, dtype=torch.float32, **kw)
    if factor < 1e-3:  # frequencies of up to 1 / factor radians: their 2^-50 counts as many times
        bound = bound + 2.0 ** -50 * 350 / factor * 2 * x.double().abs().amax()
    ref.check("out", out, (value, bound))


def test_more_threads_than_32_bits_count():
    """8.6 GB, a thread per pair: the index arithmetic in 64 bits; in place, against calls on a part."""
    n, d = (1 << 31) // 20 + 77, 40
    x = torch.empty(1, 1, n, d, dtype=torch.bfloat16, device="cuda").normal_()
    parts = {a: x[:, :, a:a + 200].clone() for a in (0, n // 2, n - 200)}
    p = llsa.RopeParams.like(x)
    llsa.llsa_rope(p, x, None, x, None)
    for a, y in parts.items():
        want = torch.empty_like(y)
        llsa.llsa_rope(llsa.RopeParams.like(y, pos_offset=a), y, None, want, None)
        assert torch.equal(x[:, :, a:a + 200], want), a
