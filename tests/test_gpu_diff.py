"""Differential attention on the GPU against its formulas in 64 bits: values and
gradients over types, head layouts, lengths, masks and padding, within bounds that count
roundings; plus streams, captured graphs, splits of a long axis, offsets behind 32 bits,
and a run together with rotary positions."""
import math

import pytest
import torch

import hierarchical_sparse_attention_mean_gb300 as llsa
from hierarchical_sparse_attention_mean_gb300 import build

import dense_ref
import diff_ref as ref
import grid_ref as grid

pytestmark = pytest.mark.gpu
T = {"bf16": torch.bfloat16, "fp32": torch.float32}
NAMES = ("o", "o2", "lse", "dq", "dk", "dv", "dlam")
TIMEOUT, BAD_INDEX = -9, -10


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()


def make(b, h, kv, nq, nk, d, dtype, q_len=None, k_len=None, seed=0, pad=float("nan"), lam_dtype=None):
    g = torch.Generator().manual_seed(seed * 1000 + nq * 7 + nk * 3 + d)
    x = {n: torch.randn(b, hh, nn, c, generator=g).to(T[dtype])
         for n, hh, nn, c in (("q", 2 * h, nq, d), ("k", 2 * kv, nk, d), ("v", kv, nk, 2 * d), ("dout", h, nq, 2 * d))}
    x["lam"] = (0.2 + 0.6 * torch.rand(h, generator=g)).to(T[lam_dtype or dtype])
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


def run(x, causal=False, scale=0.0, q_len=None, k_len=None):
    c = {n: t.cuda() for n, t in x.items()}
    p = llsa.DiffParams.like(c["q"], c["k"], c["lam"], causal=causal, scale=scale)
    ql, kl = lens(q_len), lens(k_len)
    full = lambda n: torch.full_like(c[n], 7.0)  # every row is written
    o, lse, o2 = llsa.diff_forward(p, c["q"], c["k"], c["v"], c["lam"], ql, kl, o=full("dout"), o2=full("dout"))
    dq, dk, dv, dlam = llsa.diff_backward(p, c["q"], c["k"], c["v"], c["lam"], o, o2, lse, c["dout"], ql, kl,
                                          full("q"), full("k"), full("v"), full("lam"))
    alone, lse_alone, none = llsa.diff_forward(p, c["q"], c["k"], c["v"], c["lam"], ql, kl)
    torch.cuda.synchronize()
    assert llsa.llsa_get_status() == 0 and none is None
    assert torch.equal(alone, o) and torch.equal(lse_alone, lse)  # o2 is no more than kept or not
    return {"o": o, "o2": o2, "lse": lse, "dq": dq, "dk": dk, "dv": dv, "dlam": dlam}


def both(x, dtype, names=NAMES, causal=False, scale=0.0, q_len=None, k_len=None):
    want = ref.attention(**x, causal=causal, scale=scale, q_len=q_len, k_len=k_len, dtype=T[dtype], lam_dtype=x["lam"].dtype)
    got = run(x, causal, scale, q_len, k_len)
    for n in names:
        ref.check(n, got[n], want[n])


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
    (2, 2, 1, 90, 140, 32, True, None, [97, 140]),
    (1, 2, 2, 90, 100, 72, True, None, [97]),
    (1, 2, 2, 150, 140, 96, False, None, None),
    (1, 2, 2, 1000, 1100, 64, False, None, None),
    (1, 1, 1, 700, 900, 128, True, None, None),
    (1, 2, 2, 383, 513, 8, False, None, None),
]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(str(v) for v in c[:6]) + ("-causal" if c[6] else "") +
                         ("-len" if c[7] or c[8] else ""))
def test_forward_and_backward(case, dtype):
    b, h, kv, nq, nk, d, causal, ql, kl = case
    both(make(b, h, kv, nq, nk, d, dtype, ql, kl), dtype, causal=causal, q_len=ql, k_len=kl)


@pytest.mark.parametrize("dtype,lam_dtype", [("bf16", "fp32"), ("fp32", "bf16")])
def test_lam_has_a_type_of_its_own(dtype, lam_dtype):
    both(make(2, 4, 2, 70, 200, 64, dtype, lam_dtype=lam_dtype), dtype)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("value", [0.0, 1.0, -1.5, 30.0])
def test_any_lam(value, dtype):
    x = make(1, 2, 2, 140, 150, 64, dtype, seed=2)
    x["lam"][:] = value
    both(x, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_equal_maps_cancel(dtype):
    """With lam 1 and both maps the same, o is a difference of equal numbers: only what one map's roundings leave."""
    x = make(1, 2, 2, 150, 300, 64, dtype, seed=4)
    x["q"][:, 2:], x["k"][:, 2:] = x["q"][:, :2], x["k"][:, :2]
    x["lam"][:] = 1.0
    got = run(x)
    assert not got["o"].any() and torch.equal(got["lse"][:, :2], got["lse"][:, 2:])
    both(x, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("amp,scale", [(8.0, 0.0), (1.0, 1.0), (0.01, 0.3)])
def test_scales(amp, scale, dtype):
    """Sharp and flat softmax: scores up to hundreds, where rows pass through many maxima."""
    x = make(1, 2, 2, 150, 400, 64, dtype, seed=3)
    x["q"] = (x["q"].float() * amp).to(T[dtype])
    # keys that grow along the sequence in one map and shrink in the other
    grow = torch.linspace(0.1, 2.0, 400)[:, None]
    x["k"] = torch.cat([x["k"][:, :2].float() * grow, x["k"][:, 2:].float() * grow.flip(0)], 1).to(T[dtype])
    both(x, dtype, scale=scale)


@pytest.mark.parametrize("dtype,d", [("bf16", 64), ("bf16", 128), ("fp32", 64), ("fp32", 128), ("bf16", 40)])
@pytest.mark.parametrize("nq,nk,h,kv", [(1, 20000, 2, 2), (2, 9000, 8, 2), (5000, 33, 2, 1)])
def test_long_axis_is_split(nq, nk, h, kv, dtype, d):
    """Few rows over many keys (and few keys under many rows): the long axis runs in parts."""
    both(make(1, h, kv, nq, nk, d, dtype, k_len=[nk - 3], seed=5), dtype, k_len=[nk - 3])


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("b,nq,nk", [(2, 0, 5), (2, 5, 0), (2, 0, 0), (0, 5, 5)])
def test_empty_sides(b, nq, nk, dtype):
    got = run(make(b, 2, 2, nq, nk, 64, dtype))
    assert got["o"].shape == (b, 2, nq, 128) and not got["o"].any() and not got["o2"].any()
    assert bool((got["lse"] == -math.inf).all())
    for n in ("dq", "dk", "dv", "dlam"):
        assert not got[n].any()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_bad_lengths_are_clamped_and_reported(dtype):
    x = {n: t.cuda() for n, t in make(2, 2, 2, 70, 80, 64, dtype).items()}
    p = llsa.DiffParams.like(x["q"], x["k"], x["lam"])
    args = (p, x["q"], x["k"], x["v"], x["lam"])
    o, lse, _ = llsa.diff_forward(*args, lens([75, 70]), lens([80, -4]))
    torch.cuda.synchronize()
    assert llsa.llsa_get_status() == BAD_INDEX
    o2, lse2, _ = llsa.diff_forward(*args, lens([70, 70]), lens([80, 0]))
    torch.cuda.synchronize()
    assert llsa.llsa_get_status() == 0
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("dtype,d", [("bf16", 64), ("bf16", 128), ("fp32", 64), ("fp32", 104)])
def test_repeats_are_bit_equal(dtype, d):
    x = make(2, 8, 2, 333, 450, d, dtype, q_len=[333, 200], k_len=[450, 77])
    a, b = (run(x, True, 0.0, [333, 200], [450, 77]) for _ in range(2))
    for n in a:
        assert torch.equal(a[n], b[n]), n


def test_gradients_against_differences():
    """Directional derivatives of the 64-bit loss sum(o dout), by central differences."""
    x = make(1, 4, 2, 50, 60, 64, "fp32", seed=9)
    got = run(x, causal=True)

    def loss(**kw):
        y = {n: t.double() for n, t in {**x, **kw}.items()}
        return float((ref.attention(y["q"], y["k"], y["v"], y["lam"], causal=True)["o"][0] * y["dout"]).sum())

    for n in ("q", "k", "v", "lam"):
        u = torch.randn(x[n].shape, generator=torch.Generator().manual_seed(1), dtype=torch.float64)
        u /= u.norm()
        h = 1e-4  # truncation h^2, cancellation 2^-53 |loss| / h: both far below the fp32 gradient's error
        diff = (loss(**{n: x[n].double() + h * u}) - loss(**{n: x[n].double() - h * u})) / (2 * h)
        g = got["d" + n].double().cpu()
        assert abs(float((g * u).sum()) - diff) <= 1e-5 * float(g.norm()) + 1e-6


@pytest.mark.parametrize("dtype,d", [("bf16", 64), ("bf16", 128), ("fp32", 64)])
def test_other_stream_and_captured_graph(dtype, d):
    """The call on a stream of its own, and captured with its backward pass and
    replayed on new inputs, gives what it gives on the current stream."""
    ql, kl = [200, 130], [190, 260]
    x = make(2, 4, 2, 200, 260, d, dtype, ql, kl)
    y = make(2, 4, 2, 200, 260, d, dtype, ql, kl, seed=4)
    want_x, want_y = run(x, True, 0.0, ql, kl), run(y, True, 0.0, ql, kl)
    c = {n: t.cuda() for n, t in x.items()}
    p = llsa.DiffParams.like(c["q"], c["k"], c["lam"], causal=True)
    a, b = lens(ql), lens(kl)

    def step():
        o, lse, o2 = llsa.diff_forward(p, c["q"], c["k"], c["v"], c["lam"], a, b, backward=True)
        return dict(zip(NAMES, (o, o2, lse, *llsa.diff_backward(p, c["q"], c["k"], c["v"], c["lam"], o, o2, lse, c["dout"], a, b))))

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


def test_two_captured_graphs_at_once():
    """Each graph has a workspace of its own, so that replays on two streams do not meet."""
    graphs, outs, wants = [], [], []
    for seed in (1, 2):
        x = make(1, 2, 1, 2, 9000, 64, "bf16", seed=seed)
        want = run(x)
        c = {n: t.cuda() for n, t in x.items()}
        p = llsa.DiffParams.like(c["q"], c["k"], c["lam"])
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            o, lse, o2 = llsa.diff_forward(p, c["q"], c["k"], c["v"], c["lam"], backward=True)
            grads = llsa.diff_backward(p, c["q"], c["k"], c["v"], c["lam"], o, o2, lse, c["dout"])
        graphs.append((g, c))
        outs.append(dict(zip(NAMES, (o, o2, lse, *grads))))
        wants.append(want)
    streams = [torch.cuda.Stream() for _ in graphs]
    torch.cuda.synchronize()
    for _ in range(5):
        for s, (g, _c) in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for got, want in zip(outs, wants):
        for n in want:
            assert torch.equal(got[n], want[n]), n


@pytest.mark.parametrize("wide", [True, False])
def test_captured_autograd_step(wide, monkeypatch):
    """Positions, attention and gradients captured on leaves of the capture's own, replayed
    on new inputs, while an eager graph of the same tensors lives."""
    if not wide:
        monkeypatch.setattr(llsa, "_WIDE_DIFF", 0)
    x, y = (make(2, 4, 2, 256, 256, 64, "bf16", seed=s) for s in (22, 23))
    c = {n: t.cuda() for n, t in x.items()}
    rope = llsa.RopeGridParams.like(c["q"], c["k"], columns=(16, 24, 24), extent=(4, 8, 8))

    def step(c):
        leaves = [c[n].detach().requires_grad_() for n in ("q", "k", "v", "lam")]
        o = llsa.diff_attention(*leaves, rope=rope)
        return (o, *torch.autograd.grad(o, leaves, c["dout"]))

    want = [[t.detach().clone() for t in step({n: t.cuda() for n, t in z.items()})] for z in (x, y)]
    alive = llsa.diff_attention(*(c[n].detach().requires_grad_() for n in ("q", "k", "v", "lam")), rope=rope)
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


@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("dtype,d,nq,nk,causal", [("bf16", 64, 130, 300, True), ("bf16", 64, 2, 9000, False), ("bf16", 128, 300, 300, False),
                                                  ("fp32", 64, 130, 300, True), ("fp32", 64, 300, 40, False), ("fp32", 72, 5, 2000, False)])
def test_calls_behind_each_other_share_workspaces(dtype, d, nq, nk, causal, captured):
    """A call's kernels start while the one before them ends; so many calls of two inputs in
    one set of workspaces and outputs, with copies of the outputs between them, give what
    each gives by itself."""
    xs = [{n: t.cuda() for n, t in make(2, 4, 2, nq, nk, d, dtype, seed=s).items()} for s in (21, 22)]
    x = xs[0]
    p = llsa.DiffParams.like(x["q"], x["k"], x["lam"], causal=causal)
    ws = [torch.empty(max(16, llsa.diff_workspace_bytes(p, op)), dtype=torch.uint8, device="cuda") for op in (llsa.OP_DIFF_FWD, llsa.OP_DIFF_BWD)]
    o, o2, lse = torch.empty_like(x["dout"]), torch.empty_like(x["dout"]), torch.empty(2, 8, nq, device="cuda")
    grads = [torch.empty_like(x[n]) for n in ("q", "k", "v", "lam")]

    def call(c):
        llsa.llsa_diff_fwd(p, c["q"], c["k"], c["v"], c["lam"], o, o2, lse, ws=ws[0])
        llsa.llsa_diff_bwd(p, c["q"], c["k"], c["v"], c["lam"], o, o2, lse, c["dout"], *grads, ws=ws[1])
        return [t.clone() for t in (o, o2, lse, *grads)]

    want = []
    for c in xs:
        want.append(call(c))
        torch.cuda.synchronize()
    if captured:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = [call(xs[i & 1]) for i in range(12)]
        graph.replay()
    else:
        got = [call(xs[i & 1]) for i in range(12)]
    torch.cuda.synchronize()
    for i, ts in enumerate(got):
        for t, w in zip(ts, want[i & 1]):
            assert torch.equal(t, w), i


@pytest.mark.parametrize("dtype,d,nq", [("bf16", 64, 300), ("bf16", 128, 300), ("bf16", 64, 1), ("fp32", 64, 300), ("fp32", 64, 2)])
def test_inputs_written_right_before_the_call(dtype, d, nq):
    """A call's first kernel may be set up while the kernel before it in the stream, whosever
    it is, still writes what the call reads: copies of all inputs, the lengths among them."""
    xs = [{n: t.cuda() for n, t in make(2, 4, 2, nq, 400, d, dtype, seed=s).items()} for s in (31, 32)]
    ks = [lens([400, 200]), lens([77, 400])]
    c, kl = {n: torch.empty_like(t) for n, t in xs[0].items()}, torch.empty_like(ks[0])
    p = llsa.DiffParams.like(c["q"], c["k"], c["lam"])
    rope = llsa.RopeGridParams(2, 8, nq, d, columns=(d // 2, d // 2), dtype=dtype)
    pos = torch.arange(2 * nq, dtype=torch.int32, device="cuda").view(nq, 2)

    def call(i):
        for n in c:
            c[n].copy_(xs[i][n])
        kl.copy_(ks[i])
        o, lse, o2 = llsa.diff_forward(p, c["q"], c["k"], c["v"], c["lam"], k_len=kl, backward=True)
        got = [o, lse, o2, *llsa.diff_backward(p, c["q"], c["k"], c["v"], c["lam"], o, o2, lse, c["dout"], k_len=kl)]
        c["q"].copy_(xs[1 - i]["q"])
        return [*got, llsa.rotary(c["q"], None, rope, pos=pos.mul(i + 1))]

    want = []
    for i in (0, 1):
        want.append(call(i))
        torch.cuda.synchronize()
    got = [call(i & 1) for i in range(20)]
    torch.cuda.synchronize()
    for i, ts in enumerate(got):
        for t, w in zip(ts, want[i & 1]):
            assert torch.equal(t, w), i


@pytest.mark.parametrize("dtype,d", [("bf16", 64), ("bf16", 128), ("fp32", 64)])
def test_waits_that_run_out_are_reported_and_leave_no_trace(dtype, d):
    """With the copying warps switched off every consumer's first wait runs out: the
    status reads TIMEOUT once, the kernels end, and the next calls are right."""
    x = make(1, 2, 2, 300, 400, d, dtype, seed=12)
    want = run(x)
    c = {n: t.cuda() for n, t in x.items()}
    p = llsa.DiffParams.like(c["q"], c["k"], c["lam"])
    args = (p, c["q"], c["k"], c["v"], c["lam"])
    for call in (lambda: llsa.diff_forward(*args),
                 lambda: llsa.diff_backward(*args, want["o"], want["o2"], want["lse"], c["dout"])):
        llsa.test_set_wait_limit(256, llsa.LLSA_TEST_NO_COPIES)
        try:
            call()
            torch.cuda.synchronize()
        finally:
            llsa.test_set_wait_limit(0, 0)
        assert llsa.llsa_get_status() == TIMEOUT
        assert llsa.llsa_get_status() == 0
    got = run(x)
    for n in got:
        assert torch.equal(got[n], want[n]), n


def test_a_given_stream_orders_the_call():
    """stream=: the work goes there, workspace included, whatever the current stream is."""
    x = {n: t.cuda() for n, t in make(1, 2, 2, 1, 20000, 64, "bf16").items()}
    p = llsa.DiffParams.like(x["q"], x["k"], x["lam"])
    want = llsa.diff_forward(p, x["q"], x["k"], x["v"], x["lam"])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = llsa.diff_forward(p, x["q"], x["k"], x["v"], x["lam"], stream=side)
    side.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_autograd_matches_the_calls(dtype):
    x = make(2, 4, 2, 64, 96, 64, dtype, seed=2)
    want = run(x, causal=True)
    leaves = [x[n].cuda().transpose(1, 2).contiguous().transpose(1, 2).requires_grad_() for n in ("q", "k", "v")]
    lam = x["lam"].cuda().requires_grad_()
    o = llsa.diff_attention(*leaves, lam, causal=True)
    grads = torch.autograd.grad(o, (*leaves, lam), x["dout"].cuda())
    assert torch.equal(o, want["o"])
    for g, n in zip(grads, ("dq", "dk", "dv", "dlam")):
        assert torch.equal(g, want[n]), n
    with torch.no_grad():
        assert torch.equal(llsa.diff_attention(*leaves, lam, causal=True), want["o"])


def test_one_lam_for_all_heads_and_expanded_values():
    """What is broadcast collects the gradients of every entry."""
    x = make(3, 2, 2, 40, 50, 64, "fp32", seed=8)
    k1, v1 = (x[n][:1].cuda().requires_grad_() for n in ("k", "v"))
    lam = x["lam"][:1].clone().cuda().requires_grad_()
    o = llsa.diff_attention(x["q"].cuda(), k1.expand(3, -1, -1, -1), v1.expand(3, -1, -1, -1), lam)
    dk, dv, dlam = torch.autograd.grad(o, (k1, v1, lam), x["dout"].cuda())
    x["k"], x["v"] = (x[n][:1].expand(3, -1, -1, -1) for n in ("k", "v"))
    x["lam"] = x["lam"][:1].expand(2)
    want = ref.attention(**x, dtype=torch.float32)
    for n, g in (("dk", dk), ("dv", dv), ("dlam", dlam)):
        value, bound = (t.sum(0, keepdim=True) for t in want[n])
        ref.check(n, g, (value, bound + 4 * 2.0 ** -24 * value.abs()))


def _columns_sum(t, pairs):
    """For each column, its value plus its partner's."""
    got = t.clone()
    for _, _, _, ia, ib in pairs:
        got[..., ia] = got[..., ib] = t[..., ia] + t[..., ib]
    return got


@pytest.mark.parametrize("extent,order,span", [((4, 8, 8), "raster", "axis"), ((1, 16, 16), "tile", "axis"), ((8, 4, 8), "raster", "dealt")])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_positions_attention_and_gradients_together(dtype, extent, order, span, monkeypatch):
    """Positions of a clip -> differential attention -> both backward passes, against the formulas in 64 bits."""
    b, h, kv, n, d, columns = 2, 4, 2, 256, 64, (16, 24, 24)
    x = make(b, h, kv, n, n, d, dtype, seed=6)
    leaves = [x[m].cuda().requires_grad_() for m in ("q", "k", "v", "lam")]
    rope = llsa.RopeGridParams.like(leaves[0], leaves[1], columns=columns, extent=extent, token_order=order, span=span)
    monkeypatch.setattr(llsa, "_WIDE_DIFF", 0)  # bf16 in bf16, as at larger sizes
    o = llsa.diff_attention(*leaves, rope=rope)
    got = dict(zip(("o", "dq", "dk", "dv", "dlam"), (o, *torch.autograd.grad(o, leaves, x["dout"].cuda()))))
    turned = llsa.rotary(leaves[0].detach(), leaves[1].detach(), rope)
    pos = grid.places(extent, None, order)[None]
    y = dict(x)
    for m, z in zip(("q", "k"), turned):  # the attention sees them rounded to the type
        ref.check(m, z, grid.turned(x[m], pos, columns, span, dtype=T[dtype]))
        y[m] = z.cpu()
    want = ref.attention(**y, dtype=T[dtype])
    for m in ("o", "dv", "dlam"):
        ref.check(m, got[m], want[m])
    u = ref.half_step(T[dtype])
    for m in ("dq", "dk"):
        value, bound = want[m]
        back, turn = grid.turned(value, pos, columns, span, inverse=True)
        # |cos|, |sin| <= 1: an error of either column of a pair reaches both, and the result is rounded once more
        bound = _columns_sum(bound, grid.pairs(columns, span, "half")) * (1 + u) + turn + u * back.abs()
        ref.check(m, got[m], (back, bound))


@pytest.mark.parametrize("given", [False, True])
@pytest.mark.parametrize("kind", ["grid", "image", "ragged image"])
@pytest.mark.parametrize("extent", [(3, 4), (40, 20)])
def test_small_steps_with_positions_stay_in_fp32(extent, kind, given):
    """bf16 is turned into fp32 and attended in it, and every result is rounded once."""
    b, h, kv, n, d = 2, 4, 2, extent[0] * extent[1], 64
    x = make(b, h, kv, n, n, d, "bf16", seed=16)
    leaves = [x[m].cuda().requires_grad_() for m in ("q", "k", "v", "lam")]
    q, k = leaves[:2]
    if kind == "grid":
        rope = llsa.RopeGridParams.like(q, k, columns=(32, 32), extent=extent)
    else:  # a ragged image has no grid: its positions go through fp32 copies
        rope = llsa.RopeParams.like(q, k, axes=2, width=extent[1] if kind == "image" else 7)
    pos = torch.randint(0, 99, (b, n, 2), generator=torch.Generator().manual_seed(3), dtype=torch.int32).cuda() if given else None
    o = llsa.diff_attention(*leaves, rope=rope, pos=pos)
    got = dict(zip(("o", "dq", "dk", "dv", "dlam"), (o, *torch.autograd.grad(o, leaves, x["dout"].cuda()))))
    y = dict(x)
    for m, z in zip(("q", "k"), llsa.rotary(q.detach().float(), k.detach().float(), rope.in_fp32(), pos=pos)):
        y[m] = z.cpu()
    # fp32 inside: the bounds of fp32 (o is rounded before D is formed: a half step of bf16 of it more), and one rounding to bf16
    want = ref.attention(**y, dtype=torch.float32, lam_dtype=torch.float32)
    u = ref.half_step(torch.bfloat16)
    D = u * (x["dout"].double().abs() * want["o"][0].abs()).sum(-1, keepdim=True)  # what that makes of D
    for m in ("o", "dv", "dlam"):
        value, bound = want[m]
        ref.check(m, got[m], (value, bound + u * value.abs()))
    P = _weights(y, h, kv)
    scale = 1 / math.sqrt(d)
    where = rope.grid(given) if kind != "ragged image" or given else None
    at = pos.cpu() if given else grid.places(extent)[None] if kind != "ragged image" else torch.stack([torch.arange(n) // 7, torch.arange(n) % 7], -1)[None]
    for m in ("dq", "dk"):
        value, bound = (t.clone() for t in want[m])
        for e in range(b):
            for hh in range(h):
                g = hh // (h // kv)
                # of both maps D carries it: D_1 through o, D_2 through nothing (o2 is fp32)
                err = scale * P[e, hh] * D[e, hh]
                if m == "dq":
                    bound[e, hh] += err @ y["k"][e, g].double().abs()
                else:
                    bound[e, g] += err.T @ y["q"][e, hh].double().abs()
        back, turn = grid.turned(value, at, (32, 32), inverse=True)
        bound = _columns_sum(bound, grid.pairs((32, 32), "axis", "half")) + turn + u * back.abs()
        ref.check(m, got[m], (back, bound))
    assert where is None or where.out_dtype == ""


def _weights(y, h, kv):
    """The first map's softmax, [batch, heads, nq, nk]."""
    q, k = y["q"][:, :h].double(), y["k"][:, :kv].double().repeat_interleave(h // kv, 1)
    return torch.softmax(q @ k.transpose(-1, -2) / math.sqrt(q.shape[-1]), -1)


@pytest.mark.parametrize("d", [64, 72])
def test_fp32_queries_and_keys_beside_bf16_values(d):
    """qk_dtype: the call of fp32 on the same values, with v, o, dout and dv rounded."""
    x = make(2, 4, 2, 70, 90, d, "bf16", [70, 33], [90, 61], seed=18)
    g = torch.Generator().manual_seed(4)
    for m in ("q", "k"):
        x[m] = x[m].float() * (1 + 0.01 * torch.randn(x[m].shape, generator=g))  # no values of bf16
    c = {n: t.cuda() for n, t in x.items()}
    a, b = lens([70, 33]), lens([90, 61])
    p = llsa.DiffParams.like(c["q"], c["k"], c["lam"], True, v=c["v"])
    assert p.qk_dtype == "fp32" and p.dtype == "bf16"
    o, lse, o2 = llsa.diff_forward(p, c["q"], c["k"], c["v"], c["lam"], a, b, backward=True)
    w = llsa.DiffParams.like(c["q"], c["k"], c["lam"], True)
    full = (c["q"], c["k"], c["v"].float(), c["lam"])
    o_w, lse_w, o2_w = llsa.diff_forward(w, *full, a, b, backward=True)
    assert o2.dtype == torch.float32 and torch.equal(o, o_w.bfloat16()) and torch.equal(lse, lse_w) and torch.equal(o2, o2_w)
    got = llsa.diff_backward(p, c["q"], c["k"], c["v"], c["lam"], o, o2, lse, c["dout"], a, b)
    want = llsa.diff_backward(w, *full, o.float(), o2, lse, c["dout"].float(), a, b)
    torch.cuda.synchronize()
    for m, y, z in zip(("dq", "dk", "dv", "dlam"), got, want):
        assert y.dtype == (torch.float32 if m in ("dq", "dk") else torch.bfloat16), m
        assert torch.equal(y, z.to(y.dtype)), m


SEVERAL = [
    # b, h, kv, nq, nk, d, causal: more pieces of work than SMs, so resident blocks take several one after the other
    (8, 16, 16, 300, 333, 64, False),
    (16, 12, 12, 200, 260, 64, True),
    (10, 16, 16, 256, 130, 64, False),
    (20, 16, 8, 70, 70, 40, True),
    (10, 16, 16, 150, 140, 128, True),
    (4, 40, 40, 260, 129, 96, False),
]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("ragged", [False, True])
@pytest.mark.parametrize("b,h,kv,nq,nk,d,causal", SEVERAL)
def test_blocks_take_several_pieces(b, h, kv, nq, nk, d, causal, ragged, dtype):
    """Also with lengths that leave pieces of every kind between the full ones:
    empty ones, ones without queries or without keys, and partial tiles."""
    ql = [(nq, 0, 1, nq - 1, nq // 2)[e % 5] for e in range(b)] if ragged else None
    kl = [(nk - 1, nk, nk // 3, 0, nk, 1, nk)[e % 7] for e in range(b)] if ragged else None
    both(make(b, h, kv, nq, nk, d, dtype, ql, kl, seed=11), dtype, causal=causal, q_len=ql, k_len=kl)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("d", [8, 64, 72, 128])
@pytest.mark.parametrize("h,kv,nq", [(1, 1, 1), (2, 2, 1), (2, 1, 1), (3, 1, 1), (4, 2, 2), (5, 1, 1), (2, 1, 4), (3, 1, 3)])
def test_few_rows(h, kv, nq, d, dtype):
    """One to nine rows per key head, where the choice of kernels changes."""
    both(make(2, h, kv, nq, 700, d, dtype, None, [700, 531], seed=13), dtype, causal=True, k_len=[700, 531])


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("d", [24, 64, 128])
@pytest.mark.parametrize("h,kv,nq", [(2, 2, 1), (2, 1, 1), (6, 2, 1), (8, 2, 1), (2, 1, 4), (8, 1, 1), (1, 1, 9), (3, 1, 3)])
def test_few_rows_over_many_keys(h, kv, nq, d, dtype):
    """One to nine rows per key head over keys that are split: in pairs, the last of an odd
    number by itself, a batch entry without keys and one whose last parts are empty."""
    kl = [2100, 0, 1200]
    both(make(3, h, kv, nq, 2100, d, dtype, None, kl, seed=14), dtype, causal=True, k_len=kl)


@pytest.mark.parametrize("cfg,ql,kl,causal", [
    ((2, 8, 2, 333, 450, 128), [333, 200], [450, 77], True),   # stages of the rows' numbers that come round
    ((2, 8, 2, 333, 450, 64), [333, 200], [450, 77], True),
    ((3, 4, 2, 500, 700, 96), [500, 200, 3], [450, 77, 700], False),
    ((3, 4, 2, 500, 700, 40), [500, 200, 3], [450, 77, 700], False),
    ((1, 2, 2, 1, 20000, 64), None, None, False),              # a ring of copies that comes round
    ((1, 4, 2, 1, 20000, 128), None, None, False),
    ((16, 12, 12, 200, 260, 64), None, None, True),            # several pieces per block
])
def test_many_repeats_are_bit_equal(cfg, ql, kl, causal):
    """A buffer that is handed on too early shows now and then: 60 runs give one result."""
    c = {n: t.cuda() for n, t in make(*cfg, "bf16", ql, kl, seed=19).items()}
    p = llsa.DiffParams.like(c["q"], c["k"], c["lam"], causal=causal)
    a, b = lens(ql), lens(kl)
    busy = torch.empty(1 << 24, device="cuda")
    want = None
    for i in range(60):
        if i % 3 == 0:
            busy.normal_()  # other contents of the caches
        o, lse, o2 = llsa.diff_forward(p, c["q"], c["k"], c["v"], c["lam"], a, b, backward=True)
        got = (o, o2, lse, *llsa.diff_backward(p, c["q"], c["k"], c["v"], c["lam"], o, o2, lse, c["dout"], a, b))
        want = want or got
        for n, x, y in zip(NAMES, got, want):
            assert torch.equal(x, y), (i, n)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("b,h,kv,nq,nk,causal,ql,kl", [
    (2, 6, 6, 700, 333, False, None, None), (3, 4, 2, 500, 600, True, [500, 0, 77], [1, 600, 300]), (2, 4, 1, 300, 200, False, None, [200, 0])])
def test_three_resident_blocks_take_everything(b, h, kv, nq, nk, causal, ql, kl, d):
    """The forward's blocks take many pieces of each kind in turn; results stay bit for bit."""
    x = make(b, h, kv, nq, nk, d, "bf16", ql, kl, seed=20)
    want = run(x, causal, 0.0, ql, kl)
    llsa.test_set_wait_limit(0, llsa.LLSA_TEST_FEW_BLOCKS)
    try:
        got = run(x, causal, 0.0, ql, kl)
    finally:
        llsa.test_set_wait_limit(0, 0)
    for n in want:
        assert torch.equal(got[n], want[n]), n


@pytest.mark.parametrize("few", [False, True])
@pytest.mark.parametrize("cfg,ql,kl,causal", [
    ((8, 16, 16, 300, 100, 64), None, None, False),
    ((8, 16, 4, 140, 128, 64), None, None, False),
    ((12, 16, 16, 260, 77, 40), [260, 3, 129] * 4, [77, 1, 50, 0] * 3, True),
    ((16, 12, 12, 200, 700, 64), None, [700, 60, 128, 1] * 4, False),  # pieces of one key tile between longer ones
])
def test_pieces_of_one_key_tile_keep_their_sums(cfg, ql, kl, causal, few):
    """The sums of a piece's rows pass from one map's warps to the other's through a place
    that the next piece uses too; with one tile of keys a piece is over soon."""
    x = make(*cfg, "bf16", ql, kl, seed=24)
    if few:
        llsa.test_set_wait_limit(0, llsa.LLSA_TEST_FEW_BLOCKS)
    try:
        c = {n: t.cuda() for n, t in x.items()}
        p = llsa.DiffParams.like(c["q"], c["k"], c["lam"], causal=causal)
        a, b = lens(ql), lens(kl)
        runs = [llsa.diff_forward(p, c["q"], c["k"], c["v"], c["lam"], a, b, backward=True) for _ in range(60)]
        torch.cuda.synchronize()
    finally:
        llsa.test_set_wait_limit(0, 0)
    assert llsa.llsa_get_status() == 0
    y = {n: t for n, t in x.items() if n != "dout"}
    want = ref.attention(**y, causal=causal, q_len=ql, k_len=kl)
    for n, t in zip(("o", "lse", "o2"), runs[0]):
        ref.check(n, t, want[n])
    for i, got in enumerate(runs[1:]):
        for s, t in zip(got, runs[0]):
            assert torch.equal(s, t), i


@pytest.mark.parametrize("b,h,kv,nq,nk,d,causal,ql,kl", [
    (1, 2, 2, 64, 64, 64, False, None, None),                        # the last block of dq sums
    (2, 4, 2, 130, 300, 64, True, [130, 61], [300, 290]),
    (1, 2, 1, 20, 9000, 64, False, None, None),                      # over parts of the keys
    (1, 2, 1, 100, 9000, 40, False, None, [8990]),
    (1, 66, 66, 20, 40, 64, False, None, None),                      # many heads
    (1, 2, 2, 1000, 1100, 64, False, None, None),                    # a kernel of its own
    (3, 3, 3, 5000, 200, 64, False, [5000, 0, 4097], None),          # and one for its parts
    (1, 2, 2, 64, 64, 128, False, None, None),
    (2, 4, 2, 130, 300, 96, True, [130, 61], [300, 290]),
    (1, 2, 1, 20, 9000, 128, False, None, None),
    (1, 2, 1, 100, 9000, 72, False, None, [8990]),
    (1, 66, 66, 20, 40, 80, False, None, None),
    (1, 4, 2, 1000, 1100, 128, True, None, None),
    (3, 3, 3, 5000, 200, 128, False, [5000, 0, 4097], None),
])
def test_lam_gradient_far_above_its_bound(b, h, kv, nq, nk, d, causal, ql, kl):
    """dout along a^2, other weights and signs per head: dlam is hundreds of times what its
    roundings may be, so a part that is lost, taken twice or given to another head shows."""
    x = make(b, h, kv, nq, nk, d, "bf16", ql, kl, seed=26, lam_dtype="fp32")
    y = {n: t for n, t in x.items() if n != "dout"}
    a2 = ref.attention(**y, causal=causal, q_len=ql, k_len=kl)["o2"][0]
    weight = torch.tensor([(1 + i % 5) * (-1) ** i for i in range(h)], dtype=torch.float64)[None, :, None, None]
    along = a2 / a2.square().mean(-1, keepdim=True).sqrt().clamp(min=1e-6)
    x["dout"] = (weight * (along + 0.25 * x["dout"].double())).to(torch.bfloat16)  # the padding stays no number
    want = ref.lam_gradient(**x, causal=causal, q_len=ql, k_len=kl)
    assert bool((want[0].abs() > 100 * want[1]).all())
    got = run(x, causal, 0.0, ql, kl)
    ref.check("dlam", got["dlam"], want)


def test_inputs_and_gradients_off_16_bytes():
    """Views into flat buffers, as a packed set of parameters gives them: copied, not refused."""
    x = make(1, 2, 2, 40, 50, 64, "bf16", seed=21)
    want = run(x)

    def off(t):  # two bytes behind a 16-byte boundary
        flat = torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")
        view = flat[1:].view(t.shape)
        view.copy_(t)
        return view.requires_grad_()

    leaves = [off(x[n]) for n in ("q", "k", "v", "lam")]
    o = llsa.diff_attention(*leaves)
    got = torch.autograd.grad(o, leaves, off(x["dout"]).detach())
    assert torch.equal(o, want["o"])
    for n, g in zip(("dq", "dk", "dv", "dlam"), got):
        assert torch.equal(g, want[n]), n


def test_a_number_for_one_head():
    """lam without a dimension, one head: its gradient comes back in its shape."""
    x = make(1, 1, 1, 30, 40, 64, "fp32", seed=22)
    lam = x["lam"][0].cuda().requires_grad_()
    o = llsa.diff_attention(x["q"].cuda(), x["k"].cuda(), x["v"].cuda(), lam)
    (g,) = torch.autograd.grad(o, lam, x["dout"].cuda())
    want = run(x)
    assert g.shape == () and torch.equal(g, want["dlam"][0]) and torch.equal(o, want["o"])


def test_types_that_do_not_go_together_are_refused():
    x = {n: t.cuda() for n, t in make(1, 2, 2, 30, 40, 64, "bf16").items()}
    for n in ("q", "k"):
        y = {**x, n: x[n].float()}
        with pytest.raises(ValueError):
            llsa.diff_attention(y["q"], y["k"], y["v"], y["lam"])
    with pytest.raises(ValueError):
        llsa.diff_attention(x["q"], x["k"], x["v"].float(), x["lam"])
    with pytest.raises(ValueError, match="lam"):
        llsa.diff_attention(x["q"], x["k"], x["v"], x["lam"].half())
    with pytest.raises(ValueError, match="v must have shape"):
        llsa.diff_attention(x["q"], x["k"], x["v"][..., :64].contiguous(), x["lam"])
    with pytest.raises(ValueError, match="lam must have shape"):
        llsa.diff_attention(x["q"], x["k"], x["v"], x["lam"].repeat(2))
    rope = llsa.RopeGridParams.like(x["q"], x["k"], columns=(64,))
    with pytest.raises(ValueError):
        llsa.diff_attention(x["q"], x["k"], x["v"], x["lam"], rope=rope)  # other tokens in q and k
    assert llsa.llsa_get_status() == 0


def test_nan_among_the_scores_stays_in_its_row():
    """A query with a NaN gets NaN in o and lse of that map; its neighbours do not."""
    for nq in (1, 130):
        x = make(1, 2, 2, nq, 200, 64, "bf16", seed=17)
        x["q"][0, 1, nq // 2, 3] = float("nan")  # first map of head 1
        c = {n: t.cuda() for n, t in x.items()}
        p = llsa.DiffParams.like(c["q"], c["k"], c["lam"])
        o, lse, o2 = llsa.diff_forward(p, c["q"], c["k"], c["v"], c["lam"], backward=True)
        bad = torch.zeros(1, 4, nq, dtype=torch.bool)
        bad[0, 1, nq // 2] = True
        assert torch.equal(lse.isnan().cpu(), bad) and not o2.isnan().any()
        assert torch.equal(o.isnan().all(-1).cpu(), bad[:, :2]) and torch.equal(o.isnan().any(-1).cpu(), bad[:, :2])


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("nq,nk,d,causal,ql,kl", [
    (140, 200, 64, False, [140, 70, 0], [200, 0, 90]),
    (140, 200, 128, True, [140, 101, 50], [100, 1, 200]),   # rows before the first key in causal order
    (1, 200, 64, False, None, [200, 0, 1]),
    (4, 300, 64, True, [4, 3, 4], [300, 300, 2]),
    (1, 9000, 64, False, None, [9000, 0, 8000]),            # parts of the keys, and their join
    (40, 9000, 64, True, [40, 7, 40], [9000, 0, 20]),
    (40, 8, 64, True, [40, 7, 40], [8, 0, 5]),
])
def test_rows_without_keys_are_zero_whatever_lam_is(nq, nk, d, causal, ql, kl, dtype):
    """A lam that is infinite or no number stays in its head, and there in the rows that see a key."""
    x = make(3, 3, 3, nq, nk, d, dtype, ql, kl, seed=25)
    c = {n: t.cuda() for n, t in x.items()}
    p = llsa.DiffParams.like(c["q"], c["k"], c["lam"], causal=causal)
    a, b = lens(ql), lens(kl)

    def call(lam):
        lam = torch.tensor(lam).to(T[dtype]).cuda()
        o, lse, o2 = llsa.diff_forward(p, c["q"], c["k"], c["v"], lam, a, b, backward=True)
        alone = llsa.diff_forward(p, c["q"], c["k"], c["v"], lam, a, b)[0]
        grads = llsa.diff_backward(p, c["q"], c["k"], c["v"], lam, o, o2, lse, c["dout"], a, b)
        torch.cuda.synchronize()
        assert llsa.llsa_get_status() == 0 and torch.equal(alone.nan_to_num(), o.nan_to_num())
        return dict(zip(NAMES, (o, o2, lse, *grads)))

    got, want = call([0.5, math.nan, math.inf]), call([0.5, 0.5, 0.5])
    none = got["lse"][:, :3] == -math.inf
    assert torch.equal(none, got["lse"][:, 3:] == -math.inf) and bool(none.any()) and not bool(none.all())
    assert not got["o"][none].any() and not got["o2"][none].any()
    assert bool(got["o"][:, 1][~none[:, 1]].isnan().all()) and not bool(got["o"][:, 2][~none[:, 2]].isfinite().any())
    assert not got["dq"][torch.cat([none, none], 1)].any()
    for e in range(3):
        for n in ("dk", "dv"):
            assert not got[n][e, :, kl[e]:].any(), n
    for n, heads in (("o", [0]), ("o2", [0, 1, 2]), ("lse", list(range(6))), ("dq", [0, 3]), ("dk", [0, 3]), ("dv", [0])):
        assert torch.equal(got[n][:, heads], want[n][:, heads]), n
    assert torch.equal(got["dlam"][0], want["dlam"][0])


def test_fp32_magnitudes():
    """Large, small and mixed values of fp32 keep their exponents."""
    x = make(1, 2, 2, 200, 150, 64, "fp32", seed=15)
    big = torch.tensor([2.0 ** 60, 2.0 ** -60]).repeat(75)[:, None]
    x["v"] = x["v"] * big
    x["q"], x["k"] = x["q"] * 2.0 ** 40, x["k"] * 2.0 ** -40
    x["dout"] = x["dout"] * 2.0 ** -20
    both(x, "fp32")


def test_offsets_behind_32_bits():
    """2^31 elements and more in k and in v; the weight lies on the last keys."""
    d, nk = 64, (1 << 24) + 77
    k = torch.zeros(1, 2, nk, d, dtype=torch.bfloat16, device="cuda")
    v = torch.zeros(1, 1, nk, 2 * d, dtype=torch.bfloat16, device="cuda")
    assert k.numel() > 1 << 31 and v.numel() > 1 << 31
    q = torch.ones(1, 2, 1, d, dtype=torch.bfloat16, device="cuda")
    lam = torch.full((1,), 0.5, device="cuda")
    k[0, 0, -3:] = 8.0                  # first map: scores 64 against 0, e^64 >> the number of keys
    k[0, 1, -1:] = 8.0                  # second map: on the last key alone
    v[0, 0, -3:] = torch.tensor([[1.0], [2.0], [4.0]], device="cuda")
    p = llsa.DiffParams.like(q, k, lam)
    o, lse, o2 = llsa.diff_forward(p, q, k, v, lam, backward=True)
    grads = llsa.diff_backward(p, q, k, v, lam, o, o2, lse, torch.ones_like(o))
    torch.cuda.synchronize()
    assert llsa.llsa_get_status() == 0
    assert torch.allclose(o.float(), torch.full_like(o, 7 / 3 - 2.0).float(), rtol=0, atol=2.0 ** -6)  # P rounded: 2^-8 of 7/3 and 4 / 2
    assert abs(float(lse[0, 0]) - (64 + math.log(3))) < 1e-3 and abs(float(lse[0, 1]) - 64) < 1e-3
    dv = grads[2][0, 0, -3:].float().cpu()
    want = torch.tensor([1 / 3, 1 / 3, 1 / 3 - 0.5])[:, None].expand(3, 2 * d)
    assert torch.allclose(dv, want, rtol=0, atol=2.0 ** -8)
    assert abs(float(grads[3]) + 4.0 * 2 * d) < 4.0 * 2 * d * 2.0 ** -7
    few = grads[2][0, 0, : nk // 2]     # a zero key's weight: e^-64 / 3 - 0.5 e^-64 = -2.67e-29
    lo, hi = float(few.min()), float(few.max())
    # the difference of two weights, each good to 2^-8 (as bf16, if it was rounded before) and 2^-15 (exp2 and lse)
    small = math.exp(-64)
    assert lo == hi and abs(lo - small * (1 / 3 - 0.5)) < small * (1 / 3 + 0.5) * (2.0 ** -8 + 2.0 ** -15)
