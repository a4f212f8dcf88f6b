"""Differential attention and rotary positions on several axes, on sizes their users have.

Four kinds of case:
  rope      positions on up to four axes (time, height, width) of q and k in one call (or, with `inverse`, of their gradients)
  forward   differential attention, (softmax(Q1 K1^T) - lam softmax(Q2 K2^T)) V: o and the log-sum-exp of both maps
  backward  its gradients dq, dk, dv, dlam, with o, the second map's output and the log-sum-exp in hand
  step      positions, differential attention and all gradients together, as a layer trains

Layout: q [batch, 2 heads, nq, d] and k [batch, 2 kv_heads, nk, d] hold the first maps' heads, then the second maps'; v
[batch, kv_heads, nk, 2d]; lam one number per head, in the type of the tensors.

Lengths: with `q_min` / `k_min` set, batch entry i holds a number of valid tokens that falls linearly from the padded
length (first entry) to that minimum (last entry); -1 means every token is valid.
"""
import math

import torch

own = False

_T = {"bf16": torch.bfloat16, "fp32": torch.float32}
_INF = float("inf")

_GRID = {"c0": 0, "c1": 0, "c2": 0, "c3": 0, "e0": 0, "e1": 0, "e2": 0, "e3": 0, "axes": 3, "span": "axis", "layout": "half",
         "order": "raster", "step": 1.0, "base": 10000.0, "scaling": "none", "factor": 1.0, "orig_len": 0}
_ROPE = {**_GRID, "packed": False, "given": False, "inverse": False}
_DIFF = {"causal": False, "q_min": -1, "k_min": -1}


def _rope(name, dtype, batch, heads, kv_heads, n, d, **kw):
    return {"name": name, "kind": "rope", "dtype": dtype, "batch": batch, "heads": heads, "kv_heads": kv_heads, "n": n,
            "d": d, **_ROPE, **kw}


def _diff(name, kind, dtype, batch, heads, kv_heads, nq, nk, d, **kw):
    return {"name": name, "kind": kind, "dtype": dtype, "batch": batch, "heads": heads, "kv_heads": kv_heads, "nq": nq,
            "nk": nk, "d": d, **_DIFF, **(_GRID if kind == "step" else {}), **kw}


def listed():
    return [
        # a clip of 16 frames of 64 x 64 tokens, every frame in tile order, an own ladder of frequencies for each axis
        _rope("rope-16x64x64-tile", "bf16", 1, 12, 12, 65536, 64, c0=16, c1=24, c2=24, e0=16, e1=64, e2=64, order="tile",
              layout="interleaved"),
        # one new token each of four sequences, its three positions given: latency alone
        _rope("rope-one-token", "bf16", 4, 12, 12, 1, 64, c0=16, c1=24, c2=24, span="head", given=True),
        # gradients of q and k on their way back to a packed projection's layout: mixed text and frames with positions per
        # batch entry, pairs dealt to the axes in turn, shared key heads, part of each head turned, odd length
        _rope("rope-grad-packed", "fp32", 2, 16, 4, 4095, 128, c0=32, c1=32, c2=32, span="dealt", scaling="wavelength", factor=8.0,
              orig_len=4096, packed=True, given=True, inverse=True),
        # self-attention of a 64 x 64 image's tokens: the headline's 12 heads of 64 columns as 6 differential ones
        _diff("fwd-64x64", "forward", "bf16", 2, 6, 6, 4096, 4096, 64),
        # image tokens against a padded batch of short conditioning sequences, the last of them empty
        _diff("fwd-cross-ragged", "forward", "bf16", 4, 6, 6, 4096, 333, 64, k_min=0),
        # one query against a whole 256 x 256 image, as a token is generated or an image pooled
        _diff("fwd-one-query", "forward", "bf16", 1, 6, 6, 1, 65536, 64),
        # a checking run in fp32, odd length
        _diff("fwd-fp32", "forward", "fp32", 2, 4, 4, 1023, 1023, 64),
        # gradients at 128 x 128 tokens: differential layers among the sparse ones
        _diff("bwd-128x128", "backward", "bf16", 1, 6, 6, 16384, 16384, 64),
        # causal order with shared key heads, wide head, odd length
        _diff("bwd-causal-shared", "backward", "bf16", 1, 8, 2, 4095, 4095, 128, causal=True),
        # a padded batch with lengths down to nothing on both sides, fp32, small head
        _diff("bwd-ragged-fp32", "backward", "fp32", 4, 4, 2, 512, 777, 40, q_min=0, k_min=0),
        # 8 x 8 tokens, fewer than a hierarchy needs: a training step, latency alone
        _diff("step-8x8", "step", "bf16", 1, 6, 6, 64, 64, 64, axes=2, c0=32, c1=32, e0=8, e1=8),
        # a training step of 4 frames of 32 x 32 tokens
        _diff("step-4x32x32", "step", "bf16", 2, 6, 6, 4096, 4096, 64, c0=16, c1=24, c2=24, e0=4, e1=32, e2=32),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def _draw_grid(rng, d, n):
    """Axes, their columns and the extents of a grid of n tokens or a few less."""
    axes = rng.choice([2, 3, 3, 3, 4])
    pairs = [1] * axes
    for _ in range(d // 2 // rng.choice([1, 1, 2]) - axes):
        pairs[rng.randrange(axes)] += 1
    got = {"axes": axes, **{"c%d" % a: 2 * pairs[a] for a in range(axes)}}
    extent, rest = [], n
    for a in range(axes - 1):
        extent.append(_log(rng, 1, max(1, int(rest ** 0.6))))
        rest = max(1, rest // extent[-1])
    extent.append(rest)
    rng.shuffle(extent)
    got.update({"e%d" % a: extent[a] for a in range(axes)})
    return got, math.prod(extent)


def draw(rng):
    kind = rng.choice(["rope", "forward", "forward", "backward", "backward", "step"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "fp32"])
    d = rng.choice([40, 64, 64, 64, 72, 96, 128, 128])
    kv = rng.choice([1, 2, 3, 4, 6])
    heads = kv * rng.choice([1, 1, 2, 4])
    batch = rng.choice([1, 1, 2, 3, 4])
    if kind == "rope":
        most = 2 * 12 * 65536 * 64 // (2 if dtype == "fp32" else 1)
        grid, n = _draw_grid(rng, d, _log(rng, 1, min(65536, most // (batch * (heads + kv) * d))))
        scaling = rng.choice(["none", "linear", "wavelength"])
        c = _rope("", dtype, batch, heads, kv, n, d, **grid, span=rng.choice(["axis", "head", "dealt"]),
                  layout=rng.choice(["half", "interleaved"]), packed=rng.random() < 0.5, given=rng.random() < 0.5,
                  inverse=rng.random() < 0.5, step=rng.choice([1.0, 0.5, 2.5]), scaling=scaling,
                  factor=1.0 if scaling == "none" else rng.uniform(1.5, 16),
                  orig_len=rng.choice([64, 4096]) if scaling == "wavelength" else 0)
    else:
        most = 16384 * 16384 * 6 * (1 if dtype == "bf16" else 1 / 32) * 64 / d * (20 / 28 if kind == "step" else 1)
        # gradients through a single key are zero, which leaves rounding noise alone to look at: more of them there
        few = 1 if kind == "forward" else 32
        nq = _log(rng, few if kind == "step" else 1, 16384)
        nk = nq if kind == "step" else _log(rng, few, 16384)
        while batch * heads * nq * nk > most:
            if batch > 1:
                batch -= 1
            elif nq >= nk and kind != "step":
                nq = (nq + 1) // 2
            else:
                nk = (nk + 1) // 2
                nq = nk if kind == "step" else nq
        grid = {}
        if kind == "step":
            grid, nq = _draw_grid(rng, d, nq)
            while nq < few:
                grid, nq = _draw_grid(rng, d, nk)
            nk = nq
        c = _diff("", kind, dtype, batch, heads, kv, nq, nk, d, causal=rng.random() < 0.3, **grid)
        if kind != "step":
            c.update(q_min=rng.choice([-1, -1, rng.randint(0, nq)]), k_min=rng.choice([-1, -1, rng.randint(few if batch == 1 else 0, nk)]))
    del c["name"]
    return c


def _lengths(case, side):
    """Valid tokens of each batch entry, or None where all are."""
    n, low, b = case["n" + side], case[side + "_min"], case["batch"]
    if low < 0:
        return None
    return [n - (n - low) * i // max(1, b - 1) if b > 1 else low for i in range(b)]


def _pairs(case):
    """(query, key) pairs of one map that the mask leaves."""
    lq = _lengths(case, "q") or [case["nq"]] * case["batch"]
    lk = _lengths(case, "k") or [case["nk"]] * case["batch"]
    if not case["causal"]:
        return sum(a * b for a, b in zip(lq, lk))
    got = 0
    for a, b in zip(lq, lk):
        first = b - a + 1  # keys that row 0 sees, before clipping to 0 .. b
        rows = max(0, min(a, b))  # the last `rows` rows see at least one key
        low = max(first, 1)
        got += (low + b) * rows // 2 if rows else 0
    return got


def work(case):
    size = 2 if case["dtype"] == "bf16" else 4
    b, h, kv, d = case["batch"], case["heads"], case["kv_heads"], case["d"]
    if case["kind"] == "rope":
        values = b * (h + kv) * case["n"] * d
        return {"bytes": 2 * values * size, "flops": 3 * values}
    q = b * h * case["nq"] * 2 * d * size
    k = b * kv * case["nk"] * 2 * d * size
    lse = b * 2 * h * case["nq"] * 4
    pairs = h * _pairs(case)
    # products per pair: both maps' scores 4 d and values 8 d; backward the scores again, dO V^T, dV, dQ and dK of both maps
    if case["kind"] == "forward":
        return {"bytes": 2 * q + 2 * k + lse, "flops": 12 * d * pairs}
    if case["kind"] == "backward":
        return {"bytes": 5 * q + 4 * k + lse, "flops": 20 * d * pairs}
    return {"bytes": 4 * q + 4 * k, "flops": 28 * d * pairs}


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    t = _T[case["dtype"]]

    def rows(b, h, n, d):
        return torch.randn((b, h, n, d), generator=g, device="cuda").to(t)

    st = {"case": case, "table": _table(case) if case["kind"] in ("rope", "step") else None,
          "params": _params(case) if own else None}
    b, h, kv, d = case["batch"], case["heads"], case["kv_heads"], case["d"]
    if case["kind"] == "rope":
        n = case["n"]
        if case["packed"]:  # the projection's layout: every token's q heads, then its k heads
            w = torch.randn((b, n, h + kv, d), generator=g, device="cuda").to(t)
            x = w.permute(0, 2, 1, 3)
            packed = torch.empty_like(w).permute(0, 2, 1, 3)
            head_major = (torch.empty((b, h, n, d), dtype=t, device="cuda"), torch.empty((b, kv, n, d), dtype=t, device="cuda"))
            if case["inverse"]:
                st["q"], st["k"] = x[:, :h].contiguous(), x[:, h:].contiguous()
                st["q_out"], st["k_out"] = packed[:, :h], packed[:, h:]
            else:
                st["q"], st["k"] = x[:, :h], x[:, h:]
                st["q_out"], st["k_out"] = head_major
        else:
            st["q"], st["k"] = rows(b, h, n, d), rows(b, kv, n, d)
            st["q_out"], st["k_out"] = torch.empty_like(st["q"]), torch.empty_like(st["k"])
        st["pos"] = None
        if case["given"]:
            st["pos"] = torch.randint(0, 200000, (b, n, case["axes"]), generator=g, device="cuda", dtype=torch.int32)
        return st
    st["q"], st["k"] = rows(b, 2 * h, case["nq"], d), rows(b, 2 * kv, case["nk"], d)
    st["v"] = rows(b, kv, case["nk"], 2 * d)
    # a layer begins between 0.2 and 0.8, and training moves each head a little
    st["lam"] = (0.2 + 0.6 * torch.rand((h,), generator=g, device="cuda")).to(t)
    for side in ("q", "k"):
        n = _lengths(case, side)
        st[side + "_len"] = None if n is None else torch.tensor(n, dtype=torch.int32, device="cuda")
    if case["kind"] != "forward":
        st["dout"] = rows(b, h, case["nq"], 2 * d)
    if case["kind"] == "backward":
        o, lse, o2 = _forward(st)
        st["o"], st["lse"], st["o2"] = o.to(t), lse, o2.to(t)
    if case["kind"] == "step":
        for x in ("q", "k", "v", "lam"):
            st[x].requires_grad_()
    return st


# ---------------------------------------------------------------- plain forms

def _columns(case):
    return [case["c%d" % a] for a in range(case["axes"])]


def _extents(case):
    return [case["e%d" % a] for a in range(case["axes"])]


def _owners(case):
    """(axis, place, ladder length) of every pair of the turned columns: the frequency is base^(-2 place / length)."""
    pairs = [c // 2 for c in _columns(case)]
    if case["span"] == "axis":
        return [(a, i, 2 * p) for a, p in enumerate(pairs) for i in range(p)]
    total = 2 * sum(pairs)
    if case["span"] == "head":
        axis = [a for a, p in enumerate(pairs) for _ in range(p)]
    else:
        left, axis = list(pairs), []
        while any(left):
            for a in range(len(left)):
                if left[a]:
                    left[a] -= 1
                    axis.append(a)
    return [(a, i, total) for i, a in enumerate(axis)]


def _members(case):
    """Columns of the two members of every pair, in the order of _owners."""
    pairs = [c // 2 for c in _columns(case)]
    if case["layout"] == "interleaved":
        return [(2 * i, 2 * i + 1) for i in range(sum(pairs))]
    if case["span"] != "axis":
        return [(i, i + sum(pairs)) for i in range(sum(pairs))]
    got, at = [], 0
    for p in pairs:
        got += [(at + i, at + i + p) for i in range(p)]
        at += 2 * p
    return got


def _places(case, n):
    """Position of token t on every axis of the grid, the last axis fastest, [n, axes]."""
    t = torch.arange(n, device="cuda")
    extent = _extents(case)
    if case["order"] == "tile":  # base-16 digits of a place in its frame are (row digit, column digit) pairs in base 4
        frame = extent[-1] * extent[-2]
        inside = t % frame
        k = torch.arange(8, device="cuda")
        digit = (inside[:, None] >> (4 * k)) & 15
        got = [((digit & 3) << (2 * k)).sum(-1), ((digit >> 2) << (2 * k)).sum(-1)]
        t, rest = t // frame, extent[:-2]
    else:
        got, rest = [], extent
    for e in reversed(rest):
        got.append(t % e)
        t = t // e
    return torch.stack(got[::-1], -1)


def _table(case):
    """What a layer keeps: the axis of every pair, its radians per position, the amplitude, its two columns."""
    owners = _owners(case)
    axis = torch.tensor([o[0] for o in owners], device="cuda")
    w = torch.tensor([float(case["base"]) ** (-2.0 * o[1] / o[2]) for o in owners], device="cuda", dtype=torch.float64)
    amplitude, factor = 1.0, case["factor"]
    if case["scaling"] == "linear":
        w = w / factor
    if case["scaling"] == "wavelength":
        turns = case["orig_len"] * w / (2 * math.pi)
        keep = ((turns - 1.0) / (32.0 - 1.0)).clamp(0, 1)
        w = w * (keep + (1 - keep) / factor)
        amplitude = 0.1 * math.log(factor) + 1.0
    w[axis == 0] *= case["step"]  # the first axis (time) advances by `step` from one entry to the next
    first = torch.tensor([m[0] for m in _members(case)], device="cuda")
    second = torch.tensor([m[1] for m in _members(case)], device="cuda")
    return axis, w, amplitude, first, second


def _turn(case, table, x, pos, sign):
    """x with its first columns turned by sign times their angles, in 32 bits."""
    axis, w, amplitude, first, second = table
    p = _places(case, x.shape[2])[None] if pos is None else pos
    angle = (p.double()[..., axis] * w)[:, None]
    c, s = (amplitude * angle.cos()).float(), (sign * amplitude * angle.sin()).float()
    out = x.float().clone()
    a, b = out[..., first], out[..., second]
    out[..., first], out[..., second] = a * c - b * s, a * s + b * c
    return out


def _allowed(st):
    """Which (query, key) pairs the mask leaves: [batch or 1, 1, nq, nk], or None for all."""
    case = st["case"]
    q_len, k_len = st.get("q_len"), st.get("k_len")
    if q_len is None and k_len is None and not case["causal"]:
        return None
    i = torch.arange(case["nq"], device="cuda")[None, :, None]
    j = torch.arange(case["nk"], device="cuda")[None, None, :]
    lq = torch.full((1,), case["nq"], device="cuda") if q_len is None else q_len
    lk = torch.full((1,), case["nk"], device="cuda") if k_len is None else k_len
    lq, lk = lq[:, None, None], lk[:, None, None]
    ok = (i < lq) & (j < lk)
    if case["causal"]:
        ok = ok & (j <= i + lk - lq)
    return ok[:, None]


def _probabilities(st, q, k):
    """Softmax of one map's masked logits and its log-sum-exp, [batch, kv_heads, group, nq, nk]; rows without a key are 0 and -inf."""
    s = torch.matmul(q, k.transpose(-1, -2))
    s *= 1 / math.sqrt(q.shape[-1])
    ok = _allowed(st)
    if ok is not None:
        s.masked_fill_(~ok[:, None], -_INF)
    m = s.amax(-1, keepdim=True)
    m.masked_fill_(m == -_INF, 0.0)
    s -= m
    s.exp_()
    z = s.sum(-1, keepdim=True)
    lse = (m + z.log()).squeeze(-1)
    s /= z.masked_fill(z == 0, 1.0)
    return s, lse


def _maps(x, kv):
    """[batch, 2 heads, n, d] as the two maps' 32-bit [batch, kv_heads, heads / kv_heads, n, d]."""
    return tuple(y.float().unflatten(1, (kv, -1)) for y in x.chunk(2, 1))


def _forward(st):
    """o, the log-sum-exp and the second map's output, in 32 bits."""
    kv = st["case"]["kv_heads"]
    v = st["v"].float()[:, :, None]
    outs, lses = [], []
    for q, k in zip(_maps(st["q"], kv), _maps(st["k"], kv)):
        p, lse = _probabilities(st, q, k)
        outs.append(torch.matmul(p, v).flatten(1, 2))
        lses.append(lse.flatten(1, 2))
        del p
    lam = st["lam"].float()[None, :, None, None]
    return outs[0] - lam * outs[1], torch.cat(lses, 1), outs[1]


def _gradients(st, q, k, v, lam, dout):
    """o, dq, dk, dv, dlam in 32 bits, from [batch, 2 heads or 2 kv_heads, n, d] q and k."""
    kv = st["case"]["kv_heads"]
    v = v.float()[:, :, None]
    g = dout.float().unflatten(1, (kv, -1))
    lam5 = lam.float().unflatten(0, (kv, -1))[None, :, :, None, None]
    weights = (1.0, -lam5)
    d_any = torch.matmul(g, v.transpose(-1, -2))
    o, dv, dq, dk, dlam = 0.0, 0.0, [], [], None
    for i, (qi, ki) in enumerate(zip(_maps(q, kv), _maps(k, kv))):
        p, _ = _probabilities(st, qi, ki)
        out = torch.matmul(p, v)
        o = o + weights[i] * out
        if i == 1:
            dlam = -(g.double() * out.double()).sum((0, 3, 4)).flatten()
        dv = dv + torch.matmul(p.transpose(-1, -2), weights[i] * g).sum(2)
        ds = d_any * p
        p *= ds.sum(-1, keepdim=True)
        ds -= p
        ds *= weights[i] / math.sqrt(qi.shape[-1])
        dq.append(torch.matmul(ds, ki).flatten(1, 2))
        dk.append(torch.matmul(ds.transpose(-1, -2), qi).sum(2))
        del p, ds
    return o.flatten(1, 2), torch.cat(dq, 1), torch.cat(dk, 1), dv, dlam


def _plain(st):
    case = st["case"]
    t = st["q"].dtype
    if case["kind"] == "rope":
        sign = -1.0 if case["inverse"] else 1.0
        st["q_out"].copy_(_turn(case, st["table"], st["q"], st["pos"], sign))
        st["k_out"].copy_(_turn(case, st["table"], st["k"], st["pos"], sign))
        return st["q_out"], st["k_out"]
    if case["kind"] == "forward":
        o, lse, _ = _forward(st)
        return o.to(t), lse
    if case["kind"] == "backward":
        got = _gradients(st, st["q"], st["k"], st["v"], st["lam"], st["dout"])
        return tuple(x.to(t) for x in got[1:])
    with torch.no_grad():
        q, k = (_turn(case, st["table"], st[x], None, 1.0) for x in "qk")
        o, dq, dk, dv, dlam = _gradients(st, q, k, st["v"], st["lam"], st["dout"])
        dq, dk = (_turn(case, st["table"], x, None, -1.0) for x in (dq, dk))
        return tuple(x.to(t) for x in (o, dq, dk, dv, dlam))


# ------------------------------------------------------ the framework's calls

def _grid_params(llsa, case, n, heads, kv_heads):
    axes = case["axes"]
    return llsa.RopeGridParams(case["batch"], heads, n, case["d"], kv_heads=kv_heads, columns=tuple(_columns(case)),
                               extent=None if case.get("given") else tuple(_extents(case)), span=case["span"],
                               step=(case["step"],) + (1.0,) * (axes - 1), layout=case["layout"], token_order=case["order"],
                               base=case["base"], scaling=case["scaling"], factor=case["factor"], orig_len=case["orig_len"],
                               dtype=case["dtype"])


def _params(case):
    """The description of the call that a layer keeps."""
    import hierarchical_sparse_attention_mean_gb300 as llsa
    if case["kind"] == "rope":
        return _grid_params(llsa, case, case["n"], case["heads"], case["kv_heads"])
    if case["kind"] == "step":
        return _grid_params(llsa, case, case["nq"], 2 * case["heads"], 2 * case["kv_heads"])
    return llsa.DiffParams(case["batch"], case["heads"], case["nq"], case["nk"], case["d"], kv_heads=case["kv_heads"],
                           causal=case["causal"], dtype=case["dtype"], lam_dtype=case["dtype"])


def _call(st):
    import hierarchical_sparse_attention_mean_gb300 as llsa
    case, p = st["case"], st["params"]
    if case["kind"] == "rope":
        llsa.llsa_rope_grid(p, st["q"], st["k"], st["q_out"], st["k_out"], pos=st["pos"], inverse=case["inverse"])
        return st["q_out"], st["k_out"]
    if case["kind"] == "step":
        o = llsa.diff_attention(st["q"], st["k"], st["v"], st["lam"], causal=case["causal"], rope=p)
        return (o.detach(), *torch.autograd.grad(o, (st["q"], st["k"], st["v"], st["lam"]), st["dout"]))
    if case["kind"] == "forward":
        return llsa.diff_forward(p, st["q"], st["k"], st["v"], st["lam"], q_len=st["q_len"], k_len=st["k_len"])[:2]
    return llsa.diff_backward(p, st["q"], st["k"], st["v"], st["lam"], st["o"], st["o2"], st["lse"], st["dout"],
                              q_len=st["q_len"], k_len=st["k_len"])


def run(state):
    return _call(state) if own else _plain(state)


# ------------------------------------------------------- from the definitions

def _exact_turn(case, x, pos, sign):
    """Each pair of columns as a complex number, turned on the unit circle."""
    n, axes = x.shape[2], case["axes"]
    pairs = [case["c%d" % a] // 2 for a in range(axes)]
    total = sum(pairs)
    if pos is None:
        where = []
        for t in range(n):
            at, rest = [], t
            if case["order"] == "tile":
                frame = case["e%d" % (axes - 1)] ** 2
                rest, inside = divmod(t, frame)
                r, c, place = 0, 0, 1
                while inside:
                    r, c = r + place * ((inside % 16) // 4), c + place * (inside % 4)
                    place, inside = 4 * place, inside // 16
                at = [c, r]
            for a in reversed(range(axes - len(at))):
                rest, low = divmod(rest, case["e%d" % a])
                at.append(low)
            where.append(at[::-1])
        pos = torch.tensor(where, dtype=torch.float64, device=x.device)[None]
    factor = case["factor"]
    amplitude = 0.1 * math.log(factor) + 1.0 if case["scaling"] == "wavelength" else 1.0
    out = x.double().clone()
    used = [0] * axes
    turn = 0
    for i in range(total):  # pair i, in the order of the frequencies
        if case["span"] == "dealt":
            while used[turn % axes] == pairs[turn % axes]:
                turn += 1
            axis = turn % axes
            turn += 1
        else:
            axis = next(a for a in range(axes) if used[a] < pairs[a])
        if case["span"] == "axis":
            w = case["base"] ** (-float(used[axis]) / pairs[axis])
            start = 2 * sum(pairs[:axis])
            ia = start + used[axis]
            ib = ia + pairs[axis]
        else:
            w = case["base"] ** (-float(i) / total)
            ia, ib = i, i + total
        if case["layout"] == "interleaved":
            ia, ib = 2 * i, 2 * i + 1
        used[axis] += 1
        if case["scaling"] == "linear":
            w /= factor
        if case["scaling"] == "wavelength":
            g = min(1.0, max(0.0, (case["orig_len"] * w / (2 * math.pi) - 1.0) / 31.0))
            w = g * w + (1 - g) * w / factor
        if axis == 0:
            w *= case["step"]
        z = torch.complex(x[..., ia].double(), x[..., ib].double())
        p = pos[..., axis].double()
        z = z * torch.polar(torch.full_like(p, amplitude), sign * w * p)[:, None]
        out[..., ia], out[..., ib] = z.real, z.imag
    return out


def exact(case, seed):
    kind = case["kind"]
    if kind != "rope" and case["batch"] * case["heads"] * case["nq"] * case["nk"] * case["d"] > 3e10:
        return None  # 64-bit products at that size take too long
    if kind == "rope" and case["batch"] * (case["heads"] + case["kv_heads"]) * case["n"] * case["d"] > 3e8:
        return None
    st = prepare(case, seed)
    if kind == "rope":
        sign = -1.0 if case["inverse"] else 1.0
        return tuple(_exact_turn(case, st[x], st["pos"], sign) for x in "qk")
    q, k, v, lam = (st[x].detach().double() for x in ("q", "k", "v", "lam"))
    if kind == "step":
        q, k = (_exact_turn(case, x, None, 1.0) for x in (q, k))
    b, h, kv, nq, nk, d = (case[x] for x in ("batch", "heads", "kv_heads", "nq", "nk", "d"))
    lq, lk = _lengths(case, "q") or [nq] * b, _lengths(case, "k") or [nk] * b
    o = torch.zeros((b, h, nq, 2 * d), dtype=torch.float64, device=q.device)
    dq, dk, dv, dlam = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v), torch.zeros_like(lam)
    lse = torch.full((b, 2 * h, nq), -_INF, dtype=torch.float64, device=q.device)
    for e in range(b):
        a, z = lq[e], lk[e]
        if a == 0 or z == 0:
            continue
        for head in range(h):
            key = head // (h // kv)
            V = v[e, key, :z]
            sign = {0: 1.0, 1: -float(lam[head])}
            for i in (0, 1):
                Q, K = q[e, i * h + head, :a], k[e, i * kv + key, :z]
                s = Q @ K.T / math.sqrt(d)
                if case["causal"]:
                    s = torch.where(torch.ones_like(s, dtype=torch.bool).tril(z - a), s, -_INF)
                l = torch.logsumexp(s, -1)
                lse[e, i * h + head, :a] = l
                p = torch.where(torch.isinf(l)[:, None], torch.zeros_like(s), torch.exp(s - l[:, None]))
                out = p @ V
                o[e, head, :a] += sign[i] * out
                if kind == "forward":
                    continue
                do = st["dout"][e, head, :a].double()
                if i == 1:
                    dlam[head] -= (do * out).sum()
                dp = sign[i] * do @ V.T
                ds = p * (dp - (dp * p).sum(-1, keepdim=True))
                dv[e, key, :z] += sign[i] * p.T @ do
                dq[e, i * h + head, :a] = ds @ K / math.sqrt(d)
                dk[e, i * kv + key, :z] += ds.T @ Q / math.sqrt(d)
    if kind == "forward":
        return o, lse
    if kind == "backward":
        return dq, dk, dv, dlam
    dq, dk = (_exact_turn(case, x, None, -1.0) for x in (dq, dk))
    return o, dq, dk, dv, dlam
