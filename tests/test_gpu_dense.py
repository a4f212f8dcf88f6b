"""Dense attention on the GPU against its formulas in 64 bits: values and
gradients over types, head layouts, lengths, masks and padding, within bounds
that count roundings; plus streams, captured graphs, splits of a long axis,
offsets behind 32 bits, and a run together with rotary positions."""
import math

import pytest
import torch

import hierarchical_sparse_attention_mean_gb300 as llsa
from hierarchical_sparse_attention_mean_gb300 import build

import dense_ref as ref

pytestmark = pytest.mark.gpu
T = {"bf16": torch.bfloat16, "fp32": torch.float32}
TIMEOUT, BAD_INDEX = -9, -10


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()


def make(b, h, kv, nq, nk, d, dtype, q_len=None, k_len=None, seed=0, pad=float("nan")):
    g = torch.Generator().manual_seed(seed * 1000 + nq * 7 + nk * 3 + d)
    x = {n: torch.randn(b, hh, nn, d, generator=g).to(T[dtype])
         for n, hh, nn in (("q", h, nq), ("k", kv, nk), ("v", kv, nk), ("dout", h, nq))}
    for e in range(b):  # what lies behind the lengths must not matter
        if q_len is not None:
            x["q"][e, :, q_len[e]:] = pad
            x["dout"][e, :, q_len[e]:] = pad
        if k_len is not None:
            x["k"][e, :, k_len[e]:] = pad
            x["v"][e, :, k_len[e]:] = -pad
    return x


def lens(x):
    return None if x is None else torch.tensor(x, dtype=torch.int32, device="cuda")


def run(x, causal=False, scale=0.0, q_len=None, k_len=None, dtype="bf16"):
    c = {n: t.cuda() for n, t in x.items()}
    p = llsa.DenseParams.like(c["q"], c["k"], causal=causal, scale=scale)
    ql, kl = lens(q_len), lens(k_len)
    o, lse = llsa.dense_forward(p, c["q"], c["k"], c["v"], ql, kl,
                                o=torch.full_like(c["q"], 7.0))  # every row is written
    full = [torch.full_like(c[n], 7.0) for n in ("q", "k", "v")]
    dq, dk, dv = llsa.dense_backward(p, c["q"], c["k"], c["v"], o, lse, c["dout"], ql, kl, *full)
    torch.cuda.synchronize()
    assert llsa.llsa_get_status() == 0
    return {"o": o, "lse": lse, "dq": dq, "dk": dk, "dv": dv}


CASES = [
    # b, h, kv, nq, nk, d, causal, q_len, k_len
    (1, 1, 1, 1, 1, 8, False, None, None),
    (2, 3, 3, 5, 1, 64, False, None, None),
    (1, 2, 1, 1, 300, 64, False, None, None),             # one token, shared keys
    (2, 8, 2, 3, 67, 128, True, None, None),
    (1, 2, 2, 64, 64, 64, False, None, None),
    (1, 2, 2, 128, 128, 64, True, None, None),
    (1, 4, 2, 130, 129, 64, False, None, None),
    (2, 2, 2, 257, 255, 128, True, None, None),
    (1, 2, 2, 200, 77, 64, True, None, None),             # 123 rows see nothing
    (1, 2, 1, 77, 200, 64, True, None, None),
    (1, 6, 2, 100, 150, 64, True, None, None),            # tiles run over the ends of heads
    (1, 6, 2, 100, 150, 128, True, [61], [149]),
    (1, 8, 1, 17, 90, 64, False, [9], None),              # padding inside a tile, head after head
    (3, 2, 2, 140, 190, 64, False, [140, 65, 1], [190, 1, 129]),
    (3, 2, 2, 140, 190, 64, True, [140, 65, 0], [100, 0, 190]),
    (2, 4, 4, 300, 333, 64, False, None, [333, 0]),       # one entry without keys
    (2, 2, 1, 260, 270, 128, False, [0, 259], [270, 131]),
    (1, 2, 2, 90, 100, 40, False, None, None),
    (1, 2, 2, 90, 100, 72, True, None, [97]),
    (1, 2, 2, 150, 140, 96, False, None, None),
    (1, 2, 1, 70, 90, 136, True, None, None),             # behind 128 columns
    (1, 1, 1, 40, 65, 256, False, [33], [64]),
    (2, 4, 2, 150, 270, 256, True, [150, 77], [201, 270]),
    (1, 2, 1, 300, 333, 192, False, None, [260]),
    (1, 2, 2, 1000, 1100, 64, False, None, None),
    (1, 1, 1, 700, 900, 128, True, None, None),
]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(str(v) for v in c[:6]) + ("-causal" if c[6] else "") +
                         ("-len" if c[7] or c[8] else ""))
def test_forward_and_backward(case, dtype):
    b, h, kv, nq, nk, d, causal, ql, kl = case
    x = make(b, h, kv, nq, nk, d, dtype, ql, kl)
    want = ref.attention(**x, causal=causal, q_len=ql, k_len=kl, dtype=T[dtype])
    got = run(x, causal, 0.0, ql, kl, dtype)
    for n in ("o", "lse", "dq", "dk", "dv"):
        ref.check(n, got[n], want[n])


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("amp,scale", [(8.0, 0.0), (1.0, 1.0), (0.01, 0.3)])
def test_scales(amp, scale, dtype):
    """Sharp and flat softmax: scores up to hundreds, where rows pass through many maxima."""
    x = make(1, 2, 2, 150, 400, 64, dtype, seed=3)
    x["q"] = (x["q"].float() * amp).to(T[dtype])
    # keys that grow along the sequence: the maximum keeps moving
    x["k"] = (x["k"].float() * torch.linspace(0.1, 2.0, 400)[:, None]).to(T[dtype])
    want = ref.attention(**x, scale=scale, dtype=T[dtype])
    got = run(x, scale=scale, dtype=dtype)
    for n in ("o", "lse", "dq", "dk", "dv"):
        ref.check(n, got[n], want[n])


@pytest.mark.parametrize("dtype,d", [("bf16", 64), ("bf16", 128), ("fp32", 64), ("fp32", 128), ("bf16", 200)])
@pytest.mark.parametrize("nq,nk,h,kv", [(1, 20000, 2, 2), (2, 9000, 8, 2), (5000, 33, 2, 1)])
def test_long_axis_is_split(nq, nk, h, kv, dtype, d):
    """Few rows over many keys (and few keys under many rows): the long axis runs in parts."""
    x = make(1, h, kv, nq, nk, d, dtype, k_len=[nk - 3], seed=5)
    want = ref.attention(**x, k_len=[nk - 3], dtype=T[dtype])
    got = run(x, k_len=[nk - 3], dtype=dtype)
    for n in ("o", "lse", "dq", "dk", "dv"):
        ref.check(n, got[n], want[n])


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("nq,nk", [(0, 5), (5, 0), (0, 0)])
def test_empty_sides(nq, nk, dtype):
    x = make(2, 2, 2, nq, nk, 64, dtype)
    got = run(x, dtype=dtype)
    assert got["o"].shape == (2, 2, nq, 64) and not got["o"].any()
    assert bool((got["lse"] == -math.inf).all())
    for n in ("dq", "dk", "dv"):
        assert not got[n].any()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_bad_lengths_are_clamped_and_reported(dtype):
    x = {n: t.cuda() for n, t in make(2, 2, 2, 70, 80, 64, dtype).items()}
    p = llsa.DenseParams.like(x["q"], x["k"])
    o, lse = llsa.dense_forward(p, x["q"], x["k"], x["v"], lens([75, 70]), lens([80, -4]))
    torch.cuda.synchronize()
    assert llsa.llsa_get_status() == BAD_INDEX
    o2, lse2 = llsa.dense_forward(p, x["q"], x["k"], x["v"], lens([70, 70]), lens([80, 0]))
    torch.cuda.synchronize()
    assert llsa.llsa_get_status() == 0
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("dtype,d", [("bf16", 64), ("bf16", 128), ("bf16", 256), ("fp32", 64), ("fp32", 104)])
def test_repeats_are_bit_equal(dtype, d):
    x = make(2, 8, 2, 333, 450, d, dtype, q_len=[333, 200], k_len=[450, 77])
    a, b = (run(x, True, 0.0, [333, 200], [450, 77], dtype) for _ in range(2))
    for n in a:
        assert torch.equal(a[n], b[n]), n


def test_gradients_against_differences():
    """Directional derivatives of the 64-bit loss sum(o dout), by central differences."""
    x = make(1, 4, 2, 50, 60, 64, "fp32", seed=9)
    got = run(x, causal=True, dtype="fp32")

    def loss(**kw):
        y = {n: t.double() for n, t in {**x, **kw}.items()}
        return float((ref.attention(y["q"], y["k"], y["v"], causal=True)["o"][0] * y["dout"]).sum())

    for n in ("q", "k", "v"):
        u = torch.randn(x[n].shape, generator=torch.Generator().manual_seed(1), dtype=torch.float64)
        u /= u.norm()
        h = 1e-4  # truncation h^2, cancellation 2^-53 |loss| / h: both far below the fp32 gradient's error
        diff = (loss(**{n: x[n].double() + h * u}) - loss(**{n: x[n].double() - h * u})) / (2 * h)
        g = got["d" + n].double().cpu()
        assert abs(float((g * u).sum()) - diff) <= 1e-5 * float(g.norm()) + 1e-6


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_other_stream_and_captured_graph(dtype):
    """The call on a stream of its own, and captured with its backward pass and
    replayed on new inputs, gives what it gives on the current stream."""
    ql, kl = [200, 130], [190, 260]
    x = make(2, 4, 2, 200, 260, 64, dtype, ql, kl)
    y = make(2, 4, 2, 200, 260, 64, dtype, ql, kl, seed=4)
    want_x, want_y = run(x, True, 0.0, ql, kl, dtype), run(y, True, 0.0, ql, kl, dtype)
    c = {n: t.cuda() for n, t in x.items()}
    p = llsa.DenseParams.like(c["q"], c["k"], causal=True)
    a, b = lens(ql), lens(kl)

    def step():
        o, lse = llsa.dense_forward(p, c["q"], c["k"], c["v"], a, b)
        return dict(zip(("o", "lse", "dq", "dk", "dv"),
                        (o, lse, *llsa.dense_backward(p, c["q"], c["k"], c["v"], o, lse, c["dout"], a, b))))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = step()
    torch.cuda.synchronize()
    for n in got:
        assert torch.equal(got[n], want_x[n]), n
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for source, want in ((x, want_x), (y, want_y)):
        for n in c:
            c[n].copy_(source[n])
        graph.replay()
        torch.cuda.synchronize()
        for n in got:
            assert torch.equal(got[n], want[n]), n


@pytest.mark.parametrize("dtype,d,nq", [("bf16", 64, 300), ("bf16", 128, 300), ("fp32", 64, 300), ("fp32", 128, 300), ("bf16", 256, 300)])
def test_waits_that_run_out_are_reported_and_leave_no_trace(dtype, d, nq):
    """With the copying warps switched off every consumer's first wait runs out: the
    status reads TIMEOUT once, the kernels end, and the next calls are right."""
    x = make(1, 2, 2, nq, 400, d, dtype, seed=12)
    want = run(x, dtype=dtype)
    c = {n: t.cuda() for n, t in x.items()}
    p = llsa.DenseParams.like(c["q"], c["k"])
    o, lse = want["o"], want["lse"]
    for call in (lambda: llsa.dense_forward(p, c["q"], c["k"], c["v"]),
                 lambda: llsa.dense_backward(p, c["q"], c["k"], c["v"], o, lse, c["dout"])):
        llsa.test_set_wait_limit(256, llsa.LLSA_TEST_NO_COPIES)
        try:
            call()
            torch.cuda.synchronize()
        finally:
            llsa.test_set_wait_limit(0, 0)
        assert llsa.llsa_get_status() == TIMEOUT
        assert llsa.llsa_get_status() == 0
    got = run(x, dtype=dtype)
    for n in got:
        assert torch.equal(got[n], want[n]), n


def test_a_given_stream_orders_the_call():
    """stream=: the work goes there, workspace included, whatever the current stream is."""
    x = {n: t.cuda() for n, t in make(1, 2, 2, 1, 20000, 64, "bf16").items()}
    p = llsa.DenseParams.like(x["q"], x["k"])
    want, _ = llsa.dense_forward(p, x["q"], x["k"], x["v"])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    o, lse = llsa.dense_forward(p, x["q"], x["k"], x["v"], stream=side)
    side.synchronize()
    assert torch.equal(o, want)


def test_offsets_behind_32_bits():
    """2^31 elements and more in each of k and v; the weight lies on the last keys."""
    d, nk = 64, (1 << 25) + 77
    k = torch.zeros(1, 1, nk, d, dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    assert k.numel() > 1 << 31
    q = torch.ones(1, 1, 1, d, dtype=torch.bfloat16, device="cuda")
    k[0, 0, -3:] = 8.0                  # scores 64 against 0: e^64 >> the number of keys
    v[0, 0, -3:] = torch.tensor([[1.0], [2.0], [4.0]], device="cuda")
    p = llsa.DenseParams.like(q, k)
    o, lse = llsa.dense_forward(p, q, k, v)
    dq, dk, dv = llsa.dense_backward(p, q, k, v, o, lse, q)
    torch.cuda.synchronize()
    assert llsa.llsa_get_status() == 0
    # the zero keys weigh nk e^-64: nothing
    assert torch.allclose(o.float(), torch.full_like(o, 7.0 / 3).float(), rtol=2.0 ** -7, atol=0)
    assert abs(float(lse) - (64 + math.log(3))) < 1e-3
    third = torch.full((3, d), 1 / 3)
    assert torch.allclose(dv[0, 0, -3:].float().cpu(), third, rtol=2.0 ** -7, atol=0)
    # a zero key's value gets P dO = e^-64 / 3 = 5.346e-29, rounded to bf16 (exp2 and lse add 64 log2(e) 2^-23)
    few = dv[0, 0, : nk // 2]
    lo, hi = float(few.min()), float(few.max())
    assert lo == hi and abs(lo / (math.exp(-64) / 3) - 1) < 2.0 ** -8 + 2.0 ** -15


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_autograd_matches_the_calls(dtype):
    x = make(2, 4, 2, 64, 96, 64, dtype, seed=2)
    want = run(x, causal=True, dtype=dtype)
    leaves = [x[n].cuda().transpose(1, 2).contiguous().transpose(1, 2).requires_grad_() for n in ("q", "k", "v")]
    o = llsa.dense_attention(*leaves, causal=True)
    grads = torch.autograd.grad(o, leaves, x["dout"].cuda())
    assert torch.equal(o, want["o"])
    for g, n in zip(grads, ("dq", "dk", "dv")):
        assert torch.equal(g, want[n]), n


def test_shared_gradient_of_expanded_keys():
    """Keys and values broadcast over the batch collect the gradients of every entry."""
    x = make(3, 2, 2, 40, 50, 64, "fp32", seed=8)
    k1, v1 = (x[n][:1].cuda().requires_grad_() for n in ("k", "v"))
    o = llsa.dense_attention(x["q"].cuda(), k1.expand(3, -1, -1, -1), v1.expand(3, -1, -1, -1))
    dk, dv = torch.autograd.grad(o, (k1, v1), x["dout"].cuda())
    x["k"], x["v"] = (x[n][:1].expand(3, -1, -1, -1) for n in ("k", "v"))
    want = ref.attention(**x, dtype=torch.float32)
    for n, g in (("dk", dk), ("dv", dv)):
        value, bound = (t.sum(0, keepdim=True) for t in want[n])
        ref.check(n, g, (value, bound + 4 * 2.0 ** -24 * value.abs()))


@pytest.mark.parametrize("axes,width,order", [(1, 0, "raster"), (2, 16, "raster"), (2, 16, "tile")])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_rotary_attention_and_gradients_together(dtype, axes, width, order):
    """rotary positions -> attention -> both backward passes, against autograd of
    the formulas in 64 bits."""
    b, h, kv, n, d = 2, 4, 2, 256, 64
    x = make(b, h, kv, n, n, d, dtype, seed=6)
    leaves = [x[m].cuda().requires_grad_() for m in ("q", "k", "v")]
    rope = llsa.RopeParams.like(leaves[0], leaves[1], axes=axes, width=width, token_order=order)
    o = llsa.dense_attention(*leaves, rope=rope)
    got = dict(zip(("o", "dq", "dk", "dv"), (o, *torch.autograd.grad(o, leaves, x["dout"].cuda()))))
    turned = llsa.rotary(leaves[0].detach(), leaves[1].detach(), rope)
    torch.cuda.synchronize()
    t = torch.arange(n)
    if axes == 1:
        pos = t[:, None]
    elif order == "raster":
        pos = torch.stack([t // width, t % width], -1)
    else:
        pos = torch.stack([((t >> 4) >> 2) * 4 + ((t & 15) >> 2), ((t >> 4) & 3) * 4 + (t & 3)], -1)
    y = dict(x)
    for m, z in zip(("q", "k"), turned):  # the attention sees them rounded to the type
        ref.check(m, z, ref.rotary(x[m], pos[None], axes=axes, dtype=T[dtype]))
        y[m] = z.cpu()
    want = ref.attention(**y, dtype=T[dtype])
    for m in ("o", "dv"):
        ref.check(m, got[m], want[m])
    u = ref.half_step(T[dtype])
    for m in ("dq", "dk"):
        value, bound = want[m]
        back, turn = ref.rotary(value, pos[None], axes=axes, inverse=True)
        # |cos|, |sin| <= 1: an error of either column of a pair reaches both, and the result is rounded once more
        bound = _pair_sum(bound, axes) * (1 + u) + turn + u * back.abs()
        ref.check(m, got[m], (back, bound))


def _pair_sum(t, axes):
    """For each column, its value plus its partner's (half layout)."""
    seg = t.shape[-1] // axes
    s = t.unflatten(-1, (axes, 2, seg // 2))
    return (s + s.flip(-2)).flatten(-3)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_rotary_before_the_sparse_attention(dtype):
    """llsa_attention with rope= is the sparse attention of the turned q and k, and
    its gradients turned back."""
    n, d = 256 if dtype == "fp32" else 4096, 64
    x = make(1, 2, 2, n, n, d, dtype, seed=7)
    side = math.isqrt(n)
    q, k, v = (x[m].cuda().requires_grad_() for m in ("q", "k", "v"))
    rope = llsa.RopeParams.like(q, k, axes=2, width=side, token_order="tile")
    o = llsa.llsa_attention(q, k, v, topk=4, rope=rope)
    got = torch.autograd.grad(o, (q, k, v), x["dout"].cuda())
    qr, kr = (t.detach().requires_grad_() for t in llsa.rotary(q, k, rope))
    o2 = llsa.llsa_attention(qr, kr, v, topk=4)
    dqr, dkr, dv = torch.autograd.grad(o2, (qr, kr, v), x["dout"].cuda())
    dq, dk = torch.empty_like(dqr), torch.empty_like(dkr)
    llsa.llsa_rope(rope, dqr, dkr, dq, dk, inverse=True)
    assert torch.equal(o, o2)
    for a, b in zip(got, (dq, dk, dv)):
        assert torch.equal(a, b)


SEVERAL = [
    # b, h, kv, nq, nk, d, causal: more pieces of work than SMs, so resident blocks take several one after the other
    (8, 16, 16, 300, 333, 64, False),
    (16, 12, 12, 200, 260, 64, True),      # one piece per slice forward: a last round in halves
    (10, 16, 16, 256, 130, 64, False),
    (20, 16, 8, 70, 70, 40, True),
    (10, 16, 16, 150, 140, 128, True),
    (4, 40, 40, 260, 129, 96, False),
    (4, 40, 20, 130, 200, 200, True),
]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("ragged", [False, True])
@pytest.mark.parametrize("b,h,kv,nq,nk,d,causal", SEVERAL)
def test_blocks_take_several_pieces(b, h, kv, nq, nk, d, causal, ragged, dtype):
    """Also with lengths that leave pieces of every kind between the full ones:
    empty ones, ones without queries or without keys, and partial tiles."""
    ql = [(nq, 0, 1, nq - 1, nq // 2)[e % 5] for e in range(b)] if ragged else None
    kl = [(nk - 1, nk, nk // 3, 0, nk, 1, nk)[e % 7] for e in range(b)] if ragged else None
    x = make(b, h, kv, nq, nk, d, dtype, ql, kl, seed=11)
    want = ref.attention(**x, causal=causal, q_len=ql, k_len=kl, dtype=T[dtype])
    got = run(x, causal, 0.0, ql, kl, dtype)
    for n in ("o", "lse", "dq", "dk", "dv"):
        ref.check(n, got[n], want[n])


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("d", [8, 64, 128, 136, 256])
@pytest.mark.parametrize("h,kv,nq", [(1, 1, 1), (2, 2, 1), (2, 1, 1), (3, 1, 1), (4, 2, 2), (5, 1, 1), (2, 1, 4), (3, 1, 3)])
def test_few_rows(h, kv, nq, d, dtype):
    """One to nine rows per key head, where the choice of kernels changes."""
    x = make(2, h, kv, nq, 700, d, dtype, None, [700, 531], seed=13)
    want = ref.attention(**x, causal=True, k_len=[700, 531], dtype=T[dtype])
    got = run(x, True, 0.0, None, [700, 531], dtype)
    for n in ("o", "lse", "dq", "dk", "dv"):
        ref.check(n, got[n], want[n])


@pytest.mark.parametrize("d", [8, 24, 40, 64, 72, 128])
@pytest.mark.parametrize("nq,nk", [(127, 129), (128, 128), (129, 128), (5, 3277), (3277, 5), (1, 16384)])
def test_fp32_around_the_choice_of_kernels(nq, nk, d):
    """Pairs of a slice just below and above the number from which fp32 runs on the tensor cores."""
    x = make(1, 2, 2, nq, nk, d, "fp32", seed=14)
    want = ref.attention(**x, dtype=torch.float32)
    got = run(x, dtype="fp32")
    for n in ("o", "lse", "dq", "dk", "dv"):
        ref.check(n, got[n], want[n])


def test_fp32_magnitudes():
    """The bf16 pieces of fp32 operands keep the exponent range: large, small and mixed values."""
    x = make(1, 2, 2, 200, 150, 64, "fp32", seed=15)
    big = torch.tensor([2.0 ** 60, 2.0 ** -60]).repeat(75)[:, None]
    x["v"] = x["v"] * big
    x["q"], x["k"] = x["q"] * 2.0 ** 40, x["k"] * 2.0 ** -40
    x["dout"] = x["dout"] * 2.0 ** -20
    want = ref.attention(**x, dtype=torch.float32)
    got = run(x, dtype="fp32")
    for n in ("o", "lse", "dq", "dk", "dv"):
        ref.check(n, got[n], want[n])


@pytest.mark.parametrize("dtype,d", [("bf16", 64), ("bf16", 128), ("fp32", 64), ("fp32", 128)])
def test_two_streams_at_once(dtype, d):
    """Calls on two streams, workspaces of their own, give what they give alone."""
    xs = [make(2, 8, 4, 260, 3000, d, dtype, seed=s) for s in (20, 21)]
    want = [run(x, dtype=dtype) for x in xs]
    cs = [{n: t.cuda() for n, t in x.items()} for x in xs]
    p = llsa.DenseParams.like(cs[0]["q"], cs[0]["k"])
    streams = [torch.cuda.Stream() for _ in xs]
    got = [[], []]
    torch.cuda.synchronize()
    for _ in range(5):
        for c, st, out in zip(cs, streams, got):
            o, lse = llsa.dense_forward(p, c["q"], c["k"], c["v"], stream=st)
            # a stream may be given by its number too
            out.append((o, lse, *llsa.dense_backward(p, c["q"], c["k"], c["v"], o, lse, c["dout"], stream=st.cuda_stream)))
    torch.cuda.synchronize()
    assert llsa.llsa_get_status() == 0
    for outs, w in zip(got, want):
        for out in outs:
            for t, n in zip(out, ("o", "lse", "dq", "dk", "dv")):
                assert torch.equal(t, w[n]), n


def test_captured_autograd_step():
    """rope, attention and their gradients captured on leaves of the capture's own,
    replayed on new inputs, while an eager graph of the same tensors lives."""
    x, y = (make(2, 4, 2, 256, 256, 64, "bf16", seed=s) for s in (22, 23))
    c = {n: t.cuda() for n, t in x.items()}
    rope = llsa.RopeParams.like(c["q"], c["k"], axes=2, width=16, token_order="tile")

    def step(c):
        leaves = [c[n].detach().requires_grad_() for n in ("q", "k", "v")]
        o = llsa.dense_attention(*leaves, rope=rope)
        return (o, *torch.autograd.grad(o, leaves, c["dout"]))

    want = [[t.detach().clone() for t in step({n: t.cuda() for n, t in z.items()})] for z in (x, y)]
    alive = llsa.dense_attention(*(c[n].detach().requires_grad_() for n in ("q", "k", "v")), rope=rope)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(c)
    for z, w in zip((x, y), want):
        for n in c:
            c[n].copy_(z[n])
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, w):
            assert torch.equal(a, b)
    assert torch.equal(alive, want[0][0])


@pytest.mark.parametrize("b,h,kv,n,d", [(2, 2, 1, 2, 64), (1, 4, 2, 3, 128), (3, 3, 3, 16, 72), (1, 4, 2, 300, 8), (2, 2, 2, 129, 32)])
@pytest.mark.parametrize("causal", [False, True])
def test_rotary_attention_of_few_columns_or_tokens(b, h, kv, n, d, causal):
    """bf16 inputs with rope=: fp32 until the last rounding, against autograd of the
    formulas in 64 bits on what the fp32 turn gives."""
    x = make(b, h, kv, n, n, d, "bf16", seed=31)
    leaves = [x[m].cuda().requires_grad_() for m in ("q", "k", "v")]
    rope = llsa.RopeParams.like(leaves[0], leaves[1])
    o = llsa.dense_attention(*leaves, causal=causal, rope=rope)
    got = dict(zip(("o", "dq", "dk", "dv"), (o, *torch.autograd.grad(o, leaves, x["dout"].cuda()))))
    assert all(t.dtype == torch.bfloat16 for t in got.values())
    turned = llsa.rotary(leaves[0].detach().float(), leaves[1].detach().float(), rope.in_fp32())
    y = {m: t.float() for m, t in x.items()}
    y["q"], y["k"] = (t.cpu() for t in turned)
    want = ref.attention(**y, causal=causal, dtype=torch.float32)
    u = ref.half_step(torch.bfloat16)
    for m in ("o", "dv"):
        value, bound = want[m]
        ref.check(m, got[m], (value, bound + u * (value.abs() + bound)))
    pos = torch.arange(n)[:, None]
    for m in ("dq", "dk"):
        value, bound = want[m]
        back, turn = ref.rotary(value, pos[None], inverse=True)
        bound = _pair_sum(bound, 1) * (1 + 2.0 ** -24) + turn + 2.0 ** -24 * back.abs()  # the turn's own rounding, in fp32
        ref.check(m, got[m], (back, bound + u * (back.abs() + bound)))


@pytest.mark.parametrize("d", [8, 32, 40, 64, 72, 128, 136, 256])
@pytest.mark.parametrize("nq,nk,causal,k_len", [(300, 4, False, None), (777, 7, True, [7, 0]), (9, 20, True, None), (130, 33, False, [33, 2]),
                                                (300, 41, False, [40, 41])])
def test_fp32_few_keys(nq, nk, causal, k_len, d):
    """Many rows against a handful of keys, on both sides of where the kernels change;
    with 7 keys most rows of the causal order see none."""
    x = make(2, 4, 2, nq, nk, d, "fp32", None, k_len, seed=41)
    want = ref.attention(**x, causal=causal, k_len=k_len, dtype=torch.float32)
    got = run(x, causal, 0.0, None, k_len, "fp32")
    for n in ("o", "lse", "dq", "dk", "dv"):
        ref.check(n, got[n], want[n])


@pytest.mark.parametrize("b,h,kv,nq,nk,d,causal,ql,kl", [
    (2, 6, 6, 700, 333, 64, False, None, None),            # 36 pieces, each of them in halves
    (2, 6, 3, 300, 270, 64, True, None, None),
    (3, 4, 2, 640, 200, 64, False, [640, 0, 129], [200, 77, 0]),
    (2, 6, 6, 700, 333, 128, False, None, None),
    (3, 4, 2, 330, 200, 128, True, [330, 129, 1], [200, 77, 0]),
    (1, 8, 8, 256, 140, 96, False, None, [131]),
])
def test_blocks_take_several_halves(b, h, kv, nq, nk, d, causal, ql, kl):
    """On three blocks each block takes many halved pieces, whatever the device's number of
    SMs; what a piece gives does not depend on the block that takes it."""
    x = make(b, h, kv, nq, nk, d, "bf16", ql, kl, seed=51)
    want = run(x, causal, 0.0, ql, kl)
    ref_want = ref.attention(**x, causal=causal, q_len=ql, k_len=kl, dtype=torch.bfloat16)
    llsa.test_set_wait_limit(0, llsa.LLSA_TEST_FEW_BLOCKS)
    try:
        got = run(x, causal, 0.0, ql, kl)
    finally:
        llsa.test_set_wait_limit(0, 0)
    for n in ("o", "lse", "dq", "dk", "dv"):
        assert torch.equal(got[n], want[n]), n
        ref.check(n, got[n], ref_want[n])


def off_16_bytes(t):
    """The same values in a contiguous view that starts one element into its storage."""
    flat = torch.empty(t.numel() + 1, dtype=t.dtype, device=t.device)
    view = flat[1:].view(t.shape)
    view.copy_(t)
    assert view.is_contiguous() and view.data_ptr() % 16 != 0
    return view


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_inputs_and_gradients_off_16_bytes(dtype):
    """q, k, v and the gradient that comes in may be views into flat buffers: dense and
    sparse attention and rotary positions give what aligned copies give."""
    n = 256 if dtype == "fp32" else 4096
    x = {m: t.cuda() for m, t in make(1, 2, 2, n, n, 64, dtype, seed=61).items()}
    y = {m: off_16_bytes(t) for m, t in x.items()}
    rope = llsa.RopeParams.like(x["q"], x["k"])
    calls = [lambda q, k, v: llsa.dense_attention(q, k, v), lambda q, k, v: llsa.dense_attention(q, k, v, rope=rope),
             lambda q, k, v: llsa.llsa_attention(q, k, v, topk=4), lambda q, k, v: llsa.llsa_attention(q, k, v, topk=4, rope=rope),
             lambda q, k, v: torch.cat(llsa.rotary(q, k, rope)) + 0 * v]
    for call in calls:
        out = []
        for z in (x, y):
            leaves = [z[m].detach().requires_grad_() for m in ("q", "k", "v")]
            o = call(*leaves)
            g = z["dout"] if o.shape == z["dout"].shape else torch.cat([z["dout"]] * 2)
            out.append((o.detach(), *torch.autograd.grad(o, leaves, g)))
        for a, b in zip(*out):
            assert torch.equal(a, b)
    # the gradient's place is the engine's: a slice of a concatenation that starts with an odd number of values
    leaves = [x[m].detach().requires_grad_() for m in ("q", "k", "v")]
    lead = torch.zeros(3, dtype=x["q"].dtype, device="cuda", requires_grad=True)
    w = off_16_bytes(torch.cat([lead.detach(), x["dout"].flatten()]))
    o = llsa.dense_attention(*leaves)
    got = torch.autograd.grad(torch.cat([lead, o.flatten()]), leaves, w)
    want = torch.autograd.grad(llsa.dense_attention(*leaves), leaves, x["dout"])
    for a, b in zip(got, want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("n,d,causal", [(2048, 32, False), (1500, 24, True), (2000, 16, False)])
def test_rotary_attention_of_many_tokens_stays_in_bf16(n, d, causal):
    """Behind a handful of columns, dense_attention(rope=) on many tokens is rotary() and
    dense_attention() bit for bit, in both directions."""
    x = {m: t.cuda() for m, t in make(1, 2, 2, n, n, d, "bf16", seed=71).items()}
    rope = llsa.RopeParams.like(x["q"], x["k"])
    leaves = [x[m].requires_grad_() for m in ("q", "k", "v")]
    o = llsa.dense_attention(*leaves, causal=causal, rope=rope)
    got = torch.autograd.grad(o, leaves, x["dout"])
    qr, kr = (t.detach().requires_grad_() for t in llsa.rotary(leaves[0], leaves[1], rope))
    o2 = llsa.dense_attention(qr, kr, leaves[2], causal=causal)
    dqr, dkr, dv = torch.autograd.grad(o2, (qr, kr, leaves[2]), x["dout"])
    dq, dk = torch.empty_like(dqr), torch.empty_like(dkr)
    llsa.llsa_rope(rope, dqr, dkr, dq, dk, inverse=True)
    assert torch.equal(o, o2)
    for a, b in zip(got, (dq, dk, dv)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("n", [8, 100])
def test_rotary_attention_refuses_mixed_types(n):
    """Also where bf16 stays in fp32 in between: k, v and the positions' parameters are of q's type."""
    d = 8 if n == 100 else 64
    q, k, v = (torch.zeros(1, 2, n, d, dtype=torch.bfloat16, device="cuda") for _ in range(3))
    assert llsa._wide(q, k)
    rope = llsa.RopeParams.like(q, k)
    llsa.dense_attention(q, k, v, rope=rope)
    for args in ((q, k.float(), v), (q, k, v.float()), (q, k, v.half())):
        with pytest.raises(ValueError, match="must be torch.bfloat16"):
            llsa.dense_attention(*args, rope=rope)
    with pytest.raises(ValueError, match="must be torch.float32"):
        llsa.dense_attention(q, k, v, rope=rope.in_fp32())


@pytest.mark.parametrize("dtype,d,nq,nk", [
    ("bf16", 64, 300, 333), ("bf16", 128, 300, 333), ("bf16", 200, 300, 333), ("fp32", 64, 300, 333), ("fp32", 128, 300, 333),
    ("fp32", 136, 300, 333), ("fp32", 64, 300, 9), ("fp32", 128, 300, 9),      # a handful of keys
    ("bf16", 64, 2, 90), ("fp32", 64, 2, 90), ("bf16", 256, 4, 90),            # a handful of rows, one part
    ("bf16", 64, 2, 20000), ("fp32", 128, 2, 20000), ("bf16", 64, 100, 20000), ("fp32", 64, 100, 20000),  # keys in parts
])
def test_scores_that_are_no_numbers_show(dtype, d, nq, nk):
    """A NaN in a query makes its row's o and lse NaN and no other row's; a NaN in a key
    those of every row that sees it. -infinity stays the mark of a row without keys."""
    x = {m: t.cuda() for m, t in make(1, 2, 2, nq, nk, d, dtype, seed=81).items()}
    q, k, v = x["q"], x["k"], x["v"]
    p = llsa.DenseParams.like(q, k)
    o, lse = llsa.dense_forward(p, q, k, v)
    assert bool(torch.isfinite(o).all()) and bool(torch.isfinite(lse).all())
    clean = llsa.dense_backward(p, q, k, v, o, lse, x["dout"])
    row = nq // 2
    bad = q.clone()
    bad[0, 1, row, d - 1] = float("nan")
    o2, lse2 = llsa.dense_forward(p, bad, k, v)
    assert bool(o2[0, 1, row].isnan().all()) and bool(lse2[0, 1, row].isnan())
    for got, want in zip(llsa.dense_backward(p, bad, k, v, o2, lse2, x["dout"]), clean):
        assert bool(got[0, 1].isnan().any()) and torch.equal(got[0, 0], want[0, 0])
    o2[0, 1, row], lse2[0, 1, row] = o[0, 1, row], lse[0, 1, row]
    assert torch.equal(o2, o) and torch.equal(lse2, lse)
    bad = k.clone()
    bad[0, 0, nk - 1, 0] = float("nan")
    o2, lse2 = llsa.dense_forward(p, q, bad, v)
    assert bool(o2[0, 0].isnan().all()) and bool(lse2[0, 0].isnan().all())
    assert torch.equal(o2[0, 1], o[0, 1]) and torch.equal(lse2[0, 1], lse[0, 1])
    # causal order: rows that do not see the key stay as they were; lengths that leave nothing give -infinity
    if nq == nk - 33:
        pc = llsa.DenseParams.like(q, k, causal=True)
        o, lse = llsa.dense_forward(pc, q, k, v)
        o2, lse2 = llsa.dense_forward(pc, q, bad, v)
        assert bool(lse2[0, 0, -1].isnan()) and torch.equal(o2[0, 0, :-1], o[0, 0, :-1]) and torch.equal(lse2[0, 0, :-1], lse[0, 0, :-1])
    o2, lse2 = llsa.dense_forward(p, q, bad, v, k_len=lens([0]))
    assert not o2.any() and bool((lse2 == -math.inf).all())


@pytest.mark.parametrize("dtype,d,rows,few", [
    ("bf16", 64, 2, True), ("bf16", 64, 3, False), ("bf16", 256, 2, True), ("bf16", 256, 3, False), ("bf16", 136, 4, False),
    ("fp32", 64, 4, True), ("fp32", 64, 5, False), ("fp32", 256, 4, True), ("fp32", 256, 5, False),
])
def test_which_kernel_takes_a_handful_of_rows(dtype, d, rows, few):
    """Forward: up to two rows in bf16 and four in fp32 in one pass over the keys."""
    x = {m: t.cuda() for m, t in make(1, 2 * rows, 2, 1, 700, d, dtype, seed=91).items()}
    p = llsa.DenseParams.like(x["q"], x["k"])
    llsa.profile_reset()
    llsa.profile_enable(True)
    try:
        llsa.dense_forward(p, x["q"], x["k"], x["v"])
        torch.cuda.synchronize()
        launched = {n for n, _ in llsa.profile_read()}
    finally:
        llsa.profile_enable(False)
        llsa.profile_reset()
    assert ("dense_fwd_few" in launched) is few, launched


@pytest.mark.parametrize("dtype,d", [("bf16", 64), ("fp32", 40), ("fp32", 256), ("bf16", 136)])
@pytest.mark.parametrize("nq,nk", [(7, 0), (300, 0), (0, 300)])
def test_empty_sides_report_bad_lengths(nq, nk, dtype, d):
    """Without rows or keys the outputs are zeros and -infinity, and a length that does not fit still shows."""
    x = {m: t.cuda() for m, t in make(5, 4, 2, nq, nk, d, dtype).items()}
    p = llsa.DenseParams.like(x["q"], x["k"])
    for ql, kl, status in (([nq] * 5, [nk] * 5, 0), ([nq] * 4 + [nq + 1], None, BAD_INDEX), (None, [nk] * 4 + [-1], BAD_INDEX)):
        o, lse = llsa.dense_forward(p, x["q"], x["k"], x["v"], lens(ql), lens(kl), o=torch.full_like(x["q"], 7.0))
        assert llsa.llsa_get_status() == (status if nq else 0)   # no row: no work
        full = [torch.full_like(x[n], 7.0) for n in ("q", "k", "v")]
        llsa.dense_backward(p, x["q"], x["k"], x["v"], o, lse, x["dout"], lens(ql), lens(kl), *full)
        assert llsa.llsa_get_status() == status
        assert not o.any() and bool((lse == -math.inf).all()) and not any(t.any() for t in full)


def test_rows_behind_32_bits_on_the_tensor_cores():
    """2^31 elements and more in each of q, o, dout and dq, 130 keys; dout is zero but for the
    last 300 rows, so that those are the whole backward problem."""
    d, nk, last = 64, 130, 300
    n = (1 << 25) + 77
    q = torch.empty(1, 1, n, d, dtype=torch.bfloat16, device="cuda").normal_()
    assert q.numel() > 1 << 31
    k, v = (torch.randn(1, 1, nk, d, device="cuda").bfloat16() for _ in range(2))
    dout = torch.zeros_like(q)
    dout[:, :, -last:].normal_()
    p = llsa.DenseParams.like(q, k)
    o, lse = llsa.dense_forward(p, q, k, v)
    dq, dk, dv = llsa.dense_backward(p, q, k, v, o, lse, dout)
    torch.cuda.synchronize()
    assert llsa.llsa_get_status() == 0
    want = ref.attention(q[:, :, -last:].cpu(), k.cpu(), v.cpu(), dout[:, :, -last:].cpu())
    got = {"o": o[:, :, -last:], "lse": lse[:, :, -last:], "dq": dq[:, :, -last:], "dk": dk, "dv": dv}
    for m in got:
        ref.check(m, got[m], want[m])
    assert not dq[:, :, :-last].any()
    half = q[:, :, n // 2:n // 2 + 99]
    ref.check("o", o[:, :, n // 2:n // 2 + 99], ref.attention(half.cpu(), k.cpu(), v.cpu())["o"])


@pytest.mark.parametrize("dtype,nq,d", [("bf16", 260, 64), ("fp32", 260, 64), ("bf16", 1, 64), ("bf16", 100, 256)])
def test_two_captured_graphs_at_once(dtype, nq, d):
    """Graphs with splits and workspaces of their own, replayed side by side."""
    xs = [make(2, 8, 4, nq, 3000, d, dtype, seed=s) for s in (95, 96)]
    want = [run(x, dtype=dtype) for x in xs]
    cs = [{n: t.cuda() for n, t in x.items()} for x in xs]  # alive as long as the graphs
    p = llsa.DenseParams.like(cs[0]["q"], cs[0]["k"])
    graphs, got = [], []
    for c in cs:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            o, lse = llsa.dense_forward(p, c["q"], c["k"], c["v"])
            got.append((o, lse, *llsa.dense_backward(p, c["q"], c["k"], c["v"], o, lse, c["dout"])))
    streams = [torch.cuda.Stream() for _ in graphs]
    torch.cuda.synchronize()
    for _ in range(20):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    assert llsa.llsa_get_status() == 0
    for outs, w in zip(got, want):
        for t, n in zip(outs, ("o", "lse", "dq", "dk", "dv")):
            assert torch.equal(t, w[n]), n
