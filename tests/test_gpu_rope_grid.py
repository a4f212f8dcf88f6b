"""Rotary positions on several axes on the GPU against their definition in 64 bits."""
import pytest
import torch

import hierarchical_sparse_attention_mean_gb300 as llsa
from hierarchical_sparse_attention_mean_gb300 import build

import dense_ref as ref
import grid_ref as grid

pytestmark = pytest.mark.gpu
T = {"bf16": torch.bfloat16, "fp32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()


def rand(shape, dtype, seed):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(T[dtype])


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("inverse", [False, True])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("span", ["axis", "head", "dealt"])
@pytest.mark.parametrize("d,columns", [(64, (16, 24, 24)), (64, (64,)), (128, (32, 48, 48)), (128, (16, 16, 32, 64)), (8, (2, 2, 4)),
                                       (8, (8,)), (40, (10, 2, 6)), (72, (20, 4)), (256, (2, 100, 154)), (32, (16, 16)), (24, (2,))])
def test_columns_spans_and_layouts(d, columns, span, layout, inverse, dtype):
    b, h, kv, n = 2, 3, 2, 37
    q, k = rand((b, h, n, d), dtype, d), rand((b, kv, n, d), dtype, d + 1)
    pos = torch.randint(-5000, 5000, (b, n, len(columns)), generator=torch.Generator().manual_seed(3), dtype=torch.int32)
    qc, kc = q.cuda(), k.cuda()
    p = llsa.RopeGridParams.like(qc, kc, columns=columns, span=span, layout=layout)
    qo, ko = torch.full_like(qc, 9.0), torch.full_like(kc, 9.0)
    llsa.llsa_rope_grid(p, qc, kc, qo, ko, pos=pos.cuda(), inverse=inverse)
    torch.cuda.synchronize()
    for x, got in ((q, qo), (k, ko)):
        ref.check("out", got, grid.turned(x, pos, columns, span, layout, inverse=inverse, dtype=T[dtype]))
        assert torch.equal(got.cpu()[..., sum(columns):], x[..., sum(columns):])   # the rest is a copy
    llsa.llsa_rope_grid(p, qc, kc, qc, kc, pos=pos.cuda(), inverse=inverse)        # in place
    assert torch.equal(qc, qo) and torch.equal(kc, ko)


@pytest.mark.parametrize("extent,columns,offset,order", [
    ((5,), (16,), None, "raster"), ((3, 4, 5), (6, 6, 4), (100, -7, 3), "raster"), ((2, 3, 1, 4), (4, 4, 4, 4), None, "raster"),
    ((1, 16, 16), (4, 6, 6), None, "tile"), ((3, 16, 16), (4, 6, 6), (777777, 0, -2), "tile"), ((2, 3, 4, 4), (4, 4, 4, 4), None, "tile"),
    ((64, 64), (8, 8), None, "tile"), ((1, 1, 1), (2, 2, 2), (5, 6, 7), "raster"), ((7, 1), (8, 8), None, "raster")])
@pytest.mark.parametrize("span", ["axis", "dealt"])
def test_positions_of_a_grid(extent, columns, offset, order, span):
    pos = grid.places(extent, offset, order)
    x = rand((2, 3, len(pos), 16), "bf16", 6)
    xc = x.cuda()
    p = llsa.RopeGridParams.like(xc, columns=columns, extent=extent, offset=offset or (), token_order=order, span=span)
    got = llsa.rotary(xc, rope=p)
    ref.check("out", got, grid.turned(x, pos[None], columns, span, dtype=torch.bfloat16))
    # given, they are the same to the last bit
    assert torch.equal(got, llsa.rotary(xc, rope=llsa.RopeGridParams.like(xc, columns=columns, span=span), pos=pos.int().cuda()))


@pytest.mark.parametrize("scaling,kw", [("none", {}), ("linear", {"factor": 8.0}), ("base", {"factor": 4.0}),
                                        ("wavelength", {"factor": 8.0, "orig_len": 4096}), ("wavelength", {"factor": 0.5, "orig_len": 64}),
                                        ("wavelength", {"factor": 2.5, "orig_len": 64, "low": 0.5, "high": 4.0})])
@pytest.mark.parametrize("span", ["axis", "head"])
def test_scalings_and_steps(scaling, kw, span):
    x = rand((1, 2, 50, 64), "fp32", 1)
    xc = x.cuda()
    columns, step = (16, 24, 24), (0.125, 1.0, 3.5)
    pos = torch.stack([torch.arange(50) * f for f in (1999, 3, -40)], -1).int()
    p = llsa.RopeGridParams.like(xc, columns=columns, span=span, scaling=scaling, step=step, **kw)
    want = dict(span=span, step=step, scaling=scaling, dtype=torch.float32, **kw)
    ref.check("out", llsa.rotary(xc, rope=p, pos=pos.cuda()), grid.turned(x, pos[None], columns, **want))
    p = llsa.RopeGridParams.like(xc, columns=columns, span=span, scaling=scaling, step=step, amplitude=-0.75, **kw)
    ref.check("out", llsa.rotary(xc, rope=p, pos=pos.cuda()), grid.turned(x, pos[None], columns, amplitude=-0.75, **want))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_equal_segments_are_llsa_rope(layout, dtype):
    """One and two axes with a ladder each are the older call, bit for bit."""
    q, k = rand((2, 4, 64, 64), dtype, 2).cuda(), rand((2, 2, 64, 64), dtype, 3).cuda()
    for one, many in ((dict(pos_offset=9), dict(columns=(64,), extent=(64,), offset=(9,))),
                      (dict(axes=2, width=8), dict(columns=(32, 32), extent=(8, 8))),
                      (dict(axes=2, width=16, rot_dim=32), dict(columns=(16, 16), extent=(4, 16)))):
        a = llsa.rotary(q, k, llsa.RopeParams.like(q, k, layout=layout, **one))
        b = llsa.rotary(q, k, llsa.RopeGridParams.like(q, k, layout=layout, **many))
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_far_positions_keep_their_angles():
    x = rand((1, 1, 6, 64), "fp32", 2)
    at = torch.tensor([0, 1, 16777217, 2147483647, -2147483648, -3])
    pos = torch.stack([at, at.flip(0), at], -1)
    p = llsa.RopeGridParams.like(x.cuda(), columns=(24, 24, 16))
    ref.check("out", llsa.rotary(x.cuda(), rope=p, pos=pos.int().cuda()), grid.turned(x, pos[None], (24, 24, 16), dtype=torch.float32))


@pytest.mark.parametrize("shape", ["n", "n,axes", "b,n", "b,n,axes"])
def test_position_shapes(shape):
    b, n = 2, 9
    x = rand((b, 1, n, 32), "fp32", 4).cuda()
    base = torch.randint(0, 999, (b, n), generator=torch.Generator().manual_seed(5), dtype=torch.int32)
    pos = {"n": base[0], "n,axes": base[0][:, None], "b,n": base, "b,n,axes": base[..., None]}[shape].contiguous()
    full = (base if shape.startswith("b") else base[:1].expand(b, n))[..., None]
    got = llsa.rotary(x, rope=llsa.RopeGridParams.like(x, columns=(32,)), pos=pos.cuda())
    ref.check("out", got, grid.turned(x.cpu(), full, (32,), dtype=torch.float32))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_packed_projection_in_and_out(dtype):
    """Views of a [batch, n, heads, d] projection, both ways, the neighbours untouched."""
    b, n, h, kv, d, columns = 2, 30, 4, 2, 64, (16, 24, 20)
    w = rand((b, n, h + 2 * kv, d), dtype, 10)
    wc = w.cuda()
    v = wc.permute(0, 2, 1, 3)
    q, k = v[:, :h], v[:, h:h + kv]
    p = llsa.RopeGridParams.like(q, k, columns=columns, extent=(2, 3, 5))
    qo, ko = llsa.rotary(q, k, p)
    pos = grid.places((2, 3, 5))[None]
    u = T[dtype]
    x = w.permute(0, 2, 1, 3)
    ref.check("q", qo, grid.turned(x[:, :h], pos, columns, dtype=u))
    ref.check("k", ko, grid.turned(x[:, h:h + kv], pos, columns, dtype=u))
    back = torch.full_like(wc, 5.0)
    bv = back.permute(0, 2, 1, 3)
    llsa.llsa_rope_grid(p, qo, ko, bv[:, :h], bv[:, h:h + kv], inverse=True)
    ref.check("back", bv[:, :h], grid.turned(qo.cpu(), pos, columns, inverse=True, dtype=u))
    assert bool((bv[:, h + kv:] == 5.0).all())


def test_columns_behind_the_turned_ones_may_hold_anything():
    x = rand((1, 1, 8, 16), "bf16", 11)
    x[..., 6:] = float("inf")
    x[0, 0, 3, 9] = float("nan")
    for layout in ("half", "interleaved"):
        xc = x.cuda()
        out = llsa.rotary(xc, rope=llsa.RopeGridParams.like(xc, columns=(4, 2), layout=layout, extent=(4, 2)))
        assert bool(torch.isfinite(out[..., :6]).all())
        assert torch.equal(out.cpu()[..., 6:].view(torch.int16), x[..., 6:].view(torch.int16))


def test_autograd_is_the_inverse_turn():
    q, k = (rand((2, h, 24, 64), "fp32", 12 + h).cuda().requires_grad_() for h in (4, 2))
    p = llsa.RopeGridParams.like(q, k, columns=(16, 24, 24), extent=(2, 3, 4), span="dealt", scaling="wavelength", factor=4.0, orig_len=16)
    outs = llsa.rotary(q, k, p)
    g = [torch.randn_like(t) for t in outs]
    got = torch.autograd.grad(outs, (q, k), g)
    want = [torch.empty_like(t) for t in g]
    llsa.llsa_rope_grid(p, *g, *want, inverse=True)
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    # <R x, g> = <x, R^T g>
    outs = [o.detach() for o in outs]
    lhs = sum((o.double() * t.double()).sum() for o, t in zip(outs, g))
    rhs = sum((x.double() * t.double()).sum() for x, t in zip((q.detach(), k.detach()), got))
    size = sum((o.double().abs() * t.double().abs()).sum() for o, t in zip(outs, g))
    assert abs(float(lhs - rhs)) <= 2.0 ** -20 * float(size)


def test_other_stream_and_captured_graph():
    x = rand((1, 4, 60, 64), "bf16", 20).cuda()
    p = llsa.RopeGridParams.like(x, x, columns=(16, 24, 24), extent=(3, 4, 5))
    a, b, c, d = (torch.empty_like(x) for _ in range(4))
    llsa.llsa_rope_grid(p, x, x, a, b)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    llsa.llsa_rope_grid(p, x, x, c, d, stream=side)
    side.synchronize()
    assert torch.equal(a, c) and torch.equal(b, d)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        llsa.llsa_rope_grid(p, x, x, c, d)
    x.copy_(rand((1, 4, 60, 64), "bf16", 21))
    graph.replay()
    llsa.llsa_rope_grid(p, x, x, a, b)
    torch.cuda.synchronize()
    assert torch.equal(a, c) and torch.equal(b, d)


def test_video_tokens_in_front_of_dense_attention():
    """rope= of dense_attention takes the positions of a clip, values and gradients."""
    extent, columns, d = (4, 8, 8), (16, 24, 24), 64
    q, k, v, g = (rand((1, 2, 256, d), "fp32", 30 + i) for i in range(4))
    leaves = [t.cuda().requires_grad_() for t in (q, k, v)]
    rope = llsa.RopeGridParams.like(leaves[0], leaves[1], columns=columns, extent=extent)
    o = llsa.dense_attention(*leaves, rope=rope)
    got = torch.autograd.grad(o, leaves, g.cuda())
    qr, kr = (t.detach() for t in llsa.rotary(leaves[0], leaves[1], rope))
    parts = [t.requires_grad_() for t in (qr, kr, leaves[2].detach())]
    o2 = llsa.dense_attention(*parts)
    dq, dk, dv = torch.autograd.grad(o2, parts, g.cuda())
    back = llsa.rotary(dq, dk, rope)  # wrong way round: only the inverse gives the gradient
    assert torch.equal(o, o2) and not torch.equal(got[0], back[0])
    llsa.llsa_rope_grid(rope, dq, dk, dq, dk, inverse=True)
    for a, b in zip(got, (dq, dk, dv)):
        assert torch.equal(a, b)


def test_many_heads():
    """More heads than a grid has blocks in its second dimension."""
    q, k = rand((1, 50000, 3, 8), "fp32", 40), rand((1, 90000, 3, 8), "fp32", 41)
    p = llsa.RopeGridParams.like(q, k, columns=(2, 6), extent=(1, 3), offset=(5, -1))
    pos = grid.places((1, 3), (5, -1))[None]
    for x, got in zip((q, k), llsa.rotary(q.cuda(), k.cuda(), p)):
        ref.check("x", got, grid.turned(x, pos, (2, 6), dtype=torch.float32))


def test_more_threads_than_32_bits_count():
    """8.6 GB, a thread per pair: the index arithmetic in 64 bits; in place, against calls on a part."""
    frames, d = (1 << 31) // 20 // 1024, 40
    n = frames * 1024
    x = torch.empty(1, 1, n, d, dtype=torch.bfloat16, device="cuda").normal_()
    parts = {f: x[:, :, f * 1024:(f + 1) * 1024].clone() for f in (0, frames // 2, frames - 1)}
    kw = dict(columns=(10, 2, 6))
    llsa.llsa_rope_grid(llsa.RopeGridParams.like(x, extent=(frames, 32, 32), **kw), x, None, x, None)
    for f, y in parts.items():
        want = llsa.rotary(y, rope=llsa.RopeGridParams.like(y, extent=(1, 32, 32), offset=(f, 0, 0), **kw))
        assert torch.equal(x[:, :, f * 1024:(f + 1) * 1024], want), f


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("d,columns", [(64, (16, 24, 24)), (8, (2, 2, 4)), (40, (10, 2, 6)), (256, (2, 100, 154)), (32, (16, 16))])
def test_into_the_other_type(d, columns, layout):
    """bf16 in and fp32 out is fp32's result on the same values; fp32 in and bf16 out is that rounded."""
    x = rand((2, 3, 37, d), "bf16", d).cuda()
    pos = torch.randint(-5000, 5000, (2, 37, len(columns)), generator=torch.Generator().manual_seed(3), dtype=torch.int32).cuda()
    p = llsa.RopeGridParams.like(x, columns=columns, layout=layout)
    want = llsa.rotary(x.float(), rope=p.in_fp32(), pos=pos)
    up = torch.full((2, 3, 37, d), 7.0, device="cuda")
    llsa.llsa_rope_grid(p.to_fp32(), x, None, up, None, pos=pos)
    assert torch.equal(up, want)
    down = torch.full_like(x, 7.0)
    llsa.llsa_rope_grid(p.from_fp32(), x.float(), None, down, None, pos=pos)
    assert torch.equal(down, want.bfloat16())


@pytest.mark.parametrize("kw", [dict(pos_offset=9), dict(axes=2, width=6), dict(axes=2, width=10, rot_dim=16, layout="interleaved"),
                                dict(scaling="base", factor=3.0)])
def test_the_grid_of_one_and_two_axes(kw):
    x = rand((1, 2, 60, 32), "bf16", 5).cuda()
    p = llsa.RopeParams.like(x, **kw)
    assert torch.equal(llsa.rotary(x, rope=p), llsa.rotary(x, rope=p.grid()))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("entry", ["sparse", "dense"])
@pytest.mark.parametrize("extent,order,given", [((16, 16, 16), "raster", False), ((16, 16, 16), "tile", False), ((8, 8, 64), "raster", False), (None, "raster", True)])
def test_attention_takes_a_grid(extent, order, given, entry, dtype):
    """rope= of the sparse and of dense attention: the attention of the turned q and k, and its gradients turned back."""
    g = torch.Generator().manual_seed(41)
    q, k, v, do = (torch.randn(2, 2, 4096, 64, generator=g).to(T[dtype]).cuda() for _ in range(4))
    rope = llsa.RopeGridParams.like(q, k, columns=(16, 24, 16), extent=extent, token_order=order, span="head" if given else "axis")
    pos = torch.randint(0, 999, (2, 4096, 3), generator=g, dtype=torch.int32).cuda() if given else None

    def attend(q, k, v, **kw):
        return llsa.llsa_attention(q, k, v, topk=4, **kw) if entry == "sparse" else llsa.dense_attention(q, k, v, **kw)

    leaves = [t.detach().requires_grad_() for t in (q, k, v)]
    o = attend(*leaves, rope=rope, pos=pos)
    got = torch.autograd.grad(o, leaves, do)
    turned = [t.detach().requires_grad_() for t in (*llsa.rotary(q, k, rope, pos=pos), v)]
    where = grid.places(extent, None, order)[None] if pos is None else pos.cpu()
    for t, x in zip(turned, (q, k)):
        ref.check("turned", t, grid.turned(x.cpu(), where, (16, 24, 16), rope.span, dtype=T[dtype]))
    want = attend(*turned)
    dq, dk, dv = torch.autograd.grad(want, turned, do)
    llsa.llsa_rope_grid(rope, dq, dk, dq, dk, pos=pos, inverse=True)
    assert torch.equal(o, want)
    for a, b in zip(got, (dq, dk, dv)):
        assert torch.equal(a, b)
