"""The dense-attention and rotary-position operators on sizes their users have.

Four kinds of case:
  rope      rotary positions of q and k in one call (or, with `inverse`, of their gradients)
  forward   dense attention: o and the log-sum-exp
  backward  its gradients dq, dk, dv, with o and the log-sum-exp in hand
  step      rotary positions, attention and all gradients together, as a layer trains

Lengths: with `q_min` / `k_min` set, batch entry i holds a number of valid tokens that falls linearly from the padded
length (first entry) to that minimum (last entry); -1 means every token is valid.
"""
import math

import torch

own = False

_T = {"bf16": torch.bfloat16, "fp32": torch.float32}
_INF = float("inf")

_ROPE = {"rot": 0, "layout": "half", "axes": 1, "width": 0, "order": "raster", "offset": 0, "base": 10000.0,
         "scaling": "none", "factor": 1.0, "orig_len": 0, "packed": False, "given": False, "inverse": False}
_DENSE = {"causal": False, "q_min": -1, "k_min": -1}


def _rope(name, dtype, batch, heads, kv_heads, n, d, **kw):
    return {"name": name, "kind": "rope", "dtype": dtype, "batch": batch, "heads": heads, "kv_heads": kv_heads, "n": n,
            "d": d, **_ROPE, **kw}


def _dense(name, kind, dtype, batch, heads, kv_heads, nq, nk, d, **kw):
    return {"name": name, "kind": kind, "dtype": dtype, "batch": batch, "heads": heads, "kv_heads": kv_heads, "nq": nq,
            "nk": nk, "d": d, **_DENSE, **kw}


def listed():
    return [
        # the 256 x 256 pixel tokens of the headline workload, in tile order, each pair turned by its row or column
        _rope("rope-256x256-tile", "bf16", 1, 12, 12, 65536, 64, axes=2, width=256, order="tile", layout="interleaved"),
        # one new token far into a sequence: latency alone
        _rope("rope-one-token", "bf16", 1, 12, 12, 1, 64, offset=777777),
        # gradients of q and k on their way back to a packed projection's layout: half of each head turned, shared key
        # heads, positions given per batch entry and stretched for a context 8 times the trained one, odd length
        _rope("rope-grad-packed", "fp32", 2, 16, 4, 4095, 128, rot=64, scaling="wavelength", factor=8.0, orig_len=4096,
              packed=True, given=True, inverse=True),
        # self-attention of a 64 x 64 image's tokens
        _dense("fwd-64x64", "forward", "bf16", 2, 8, 8, 4096, 4096, 64),
        # image tokens against a padded batch of short conditioning sequences, the last of them empty
        _dense("fwd-cross-ragged", "forward", "bf16", 4, 12, 12, 4096, 333, 64, k_min=0),
        # one query that pools a whole 256 x 256 image
        _dense("fwd-one-query", "forward", "bf16", 1, 12, 12, 1, 65536, 64),
        # a checking run in fp32, odd length
        _dense("fwd-fp32", "forward", "fp32", 2, 8, 8, 1023, 1023, 64),
        # gradients at 128 x 128 tokens: dense layers among the sparse ones
        _dense("bwd-128x128", "backward", "bf16", 1, 12, 12, 16384, 16384, 64),
        # causal order with shared key heads, wide head, odd length
        _dense("bwd-causal-shared", "backward", "bf16", 1, 16, 4, 4095, 4095, 128, causal=True),
        # a padded batch with lengths down to nothing on both sides, fp32, small head
        _dense("bwd-ragged-fp32", "backward", "fp32", 4, 4, 4, 512, 777, 40, q_min=0, k_min=0),
        # 8 x 8 tokens, fewer than a hierarchy needs: a training step, latency alone
        _dense("step-8x8", "step", "bf16", 1, 12, 12, 64, 64, 64, axes=2, width=8),
        # a training step of a 64 x 64 image with two-axis rotary positions
        _dense("step-64x64", "step", "bf16", 2, 12, 12, 4096, 4096, 64, axes=2, width=64),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    kind = rng.choice(["rope", "forward", "forward", "backward", "backward", "step"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "fp32"])
    d = rng.choice([8, 40, 64, 64, 72, 96, 128, 128])
    kv = rng.choice([1, 2, 3, 4, 8])
    heads = kv * rng.choice([1, 1, 2, 4])
    batch = rng.choice([1, 1, 2, 3, 4])
    if kind == "rope":
        most = 2 * 12 * 65536 * 64 * 2 // (4 if dtype == "fp32" else 2)
        n = _log(rng, 1, min(65536, most // (batch * (heads + kv) * d)))
        axes = rng.choice([1, 2])
        scaling = rng.choice(["none", "linear", "base", "wavelength"])
        c = _rope("", dtype, batch, heads, kv, n, d, axes=axes, rot=rng.choice([0, 0, 4 * axes * max(1, d // 16)]),
                  layout=rng.choice(["half", "interleaved"]), packed=rng.random() < 0.5, given=rng.random() < 0.5,
                  inverse=rng.random() < 0.5, scaling=scaling, factor=1.0 if scaling == "none" else rng.uniform(1.5, 16),
                  orig_len=rng.choice([64, 4096]) if scaling == "wavelength" else 0, width=rng.randint(1, 300) if axes == 2 else 0,
                  offset=rng.choice([0, 0, 100000]) if axes == 1 else 0)
    else:
        most = 16384 * 16384 * 12 * (1 if dtype == "bf16" else 1 / 32) * 64 / d
        # gradients through a single key are zero, which leaves rounding noise alone to look at: two at least there
        few = 1 if kind == "forward" else 2
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
        c = _dense("", kind, dtype, batch, heads, kv, nq, nk, d, causal=rng.random() < 0.3)
        if kind == "step":
            c.update(axes=rng.choice([1, 2]), width=rng.randint(1, 128))
        else:
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
    """(query, key) pairs of one head that the mask leaves."""
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
    q = b * h * case["nq"] * d * size
    k = b * kv * case["nk"] * d * size
    lse = b * h * case["nq"] * 4
    pairs = h * _pairs(case)
    if case["kind"] == "forward":
        return {"bytes": 2 * q + 2 * k + lse, "flops": 4 * d * pairs}
    if case["kind"] == "backward":
        return {"bytes": 4 * q + 4 * k + lse, "flops": 10 * d * pairs}
    return {"bytes": 4 * q + 4 * k, "flops": 14 * d * pairs}


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    t = _T[case["dtype"]]

    def rows(b, h, n, d):
        return torch.randn((b, h, n, d), generator=g, device="cuda").to(t)

    st = {"case": case}
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
    st["q"], st["k"], st["v"] = rows(b, h, case["nq"], d), rows(b, kv, case["nk"], d), rows(b, kv, case["nk"], d)
    for side in ("q", "k"):
        n = _lengths(case, side)
        st[side + "_len"] = None if n is None else torch.tensor(n, dtype=torch.int32, device="cuda")
    if case["kind"] != "forward":
        st["dout"] = rows(b, h, case["nq"], d)
    if case["kind"] == "backward":
        st["o"], st["lse"] = _forward(st)
    if case["kind"] == "step":
        st["pos"] = None
        st["q"], st["k"], st["v"] = (x.requires_grad_() for x in (st["q"], st["k"], st["v"]))
    return st


# ---------------------------------------------------------------- plain forms

def _angles(case, n, pos):
    """Angle of each token and pair, [1 or batch, 1, n, pairs], in 64 bits, and the factor on cos and sin."""
    axes = case["axes"]
    seg = (case.get("rot") or case["d"]) // axes
    i = torch.arange(seg // 2, device="cuda", dtype=torch.float64)
    scaling, factor = case.get("scaling", "none"), case.get("factor", 1.0)
    base = case.get("base", 10000.0)
    if scaling == "base":
        base = base * factor ** (seg / (seg - 2))
    w = base ** (-2 * i / seg)
    amplitude = 1.0
    if scaling == "linear":
        w = w / factor
    if scaling == "wavelength":
        turns = case["orig_len"] * w / (2 * math.pi)
        keep = ((turns - 1.0) / (32.0 - 1.0)).clamp(0, 1)
        w = w * (keep + (1 - keep) / factor)
        amplitude = 0.1 * math.log(factor) + 1.0
    if pos is None:
        t = torch.arange(n, device="cuda")
        if axes == 1:
            p = (t + case.get("offset", 0))[:, None]
        elif case.get("order", "raster") == "raster":
            p = torch.stack([t // case["width"], t % case["width"]], -1)
        else:  # base-16 digits of a tile position are (row digit, column digit) pairs in base 4
            k = torch.arange(8, device="cuda")
            digit = (t[:, None] >> (4 * k)) & 15
            p = torch.stack([((digit >> 2) << (2 * k)).sum(-1), ((digit & 3) << (2 * k)).sum(-1)], -1)
        p = p[None]
    else:
        p = pos
    return (p.double()[..., None] * w).flatten(-2)[:, None], amplitude


def _turn(case, x, pos, sign):
    """x with its first columns turned by sign times their angles, in 32 bits."""
    axes = case["axes"]
    rot = case.get("rot") or case["d"]
    angle, amplitude = _angles(case, x.shape[2], pos)
    c, s = (amplitude * angle.cos()).float(), (sign * amplitude * angle.sin()).float()
    c, s = (y.unflatten(-1, (axes, -1)) for y in (c, s))
    head, rest = x[..., :rot].float(), x[..., rot:].float()
    if case.get("layout", "half") == "half":
        head = head.unflatten(-1, (axes, 2, -1))
        a, b = head[..., 0, :], head[..., 1, :]
        out = torch.stack([a * c - b * s, a * s + b * c], -2).flatten(-3)
    else:
        head = head.unflatten(-1, (axes, -1, 2))
        a, b = head[..., 0], head[..., 1]
        out = torch.stack([a * c - b * s, a * s + b * c], -1).flatten(-3)
    return torch.cat([out, rest], -1)


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
    """Softmax of the masked logits and its log-sum-exp, [batch, kv_heads, group, nq, nk] in 32 bits; rows without a key are 0 and -inf."""
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


def _split(st, x):
    """[batch, heads, n, d] as 32-bit [batch, kv_heads, heads / kv_heads, n, d]."""
    return x.float().unflatten(1, (st["case"]["kv_heads"], -1))


def _forward(st):
    t = st["q"].dtype
    q, k, v = (_split(st, st[x]) for x in "qkv")
    p, lse = _probabilities(st, q, k)
    return torch.matmul(p, v).flatten(1, 2).to(t), lse.flatten(1, 2)


def _gradients(st, q, k, v, dout):
    """o, dq, dk, dv in 32 bits, from [batch, kv_heads, group, n, d] inputs."""
    p, _ = _probabilities(st, q, k)
    o = torch.matmul(p, v)
    dv = torch.matmul(p.transpose(-1, -2), dout).sum(2, keepdim=True)
    ds = torch.matmul(dout, v.transpose(-1, -2))
    ds *= p
    row = ds.sum(-1, keepdim=True)
    p *= row
    ds -= p
    ds *= 1 / math.sqrt(q.shape[-1])
    dq = torch.matmul(ds, k)
    dk = torch.matmul(ds.transpose(-1, -2), q).sum(2, keepdim=True)
    return tuple(x.flatten(1, 2) for x in (o, dq, dk, dv))


def _plain(st):
    case = st["case"]
    t = st["q"].dtype
    if case["kind"] == "rope":
        sign = -1.0 if case["inverse"] else 1.0
        st["q_out"].copy_(_turn(case, st["q"], st["pos"], sign))
        st["k_out"].copy_(_turn(case, st["k"], st["pos"], sign))
        return st["q_out"], st["k_out"]
    if case["kind"] == "forward":
        return _forward(st)
    if case["kind"] == "backward":
        got = _gradients(st, *(_split(st, st[x]) for x in ("q", "k", "v", "dout")))
        return tuple(x.to(t) for x in got[1:])
    with torch.no_grad():
        q, k = (_turn(case, st[x], None, 1.0) for x in "qk")
        o, dq, dk, dv = _gradients(st, _split(st, q), _split(st, k), _split(st, st["v"]), _split(st, st["dout"]))
        dq, dk = (_turn(case, x, None, -1.0) for x in (dq, dk))
        return tuple(x.to(t) for x in (o, dq, dk, dv))


# ------------------------------------------------------ the framework's calls

def _rope_params(llsa, case, n):
    return llsa.RopeParams(case["batch"], case["heads"], n, case["d"], kv_heads=case["kv_heads"], rot_dim=case.get("rot", 0),
                           layout=case.get("layout", "half"), axes=case["axes"], width=case["width"] if case["axes"] == 2 else 0,
                           token_order=case.get("order", "raster"), pos_offset=case.get("offset", 0), base=case.get("base", 10000.0),
                           scaling=case.get("scaling", "none"), factor=case.get("factor", 1.0),
                           orig_len=case.get("orig_len", 0), dtype=case["dtype"])


def _call(st):
    import hierarchical_sparse_attention_mean_gb300 as llsa
    case = st["case"]
    if case["kind"] == "rope":
        llsa.llsa_rope(_rope_params(llsa, case, case["n"]), st["q"], st["k"], st["q_out"], st["k_out"], pos=st["pos"],
                       inverse=case["inverse"])
        return st["q_out"], st["k_out"]
    if case["kind"] == "step":
        o = llsa.dense_attention(st["q"], st["k"], st["v"], causal=case["causal"],
                                 rope=_rope_params(llsa, case, case["nq"]))
        return (o.detach(), *torch.autograd.grad(o, (st["q"], st["k"], st["v"]), st["dout"]))
    p = llsa.DenseParams(case["batch"], case["heads"], case["nq"], case["nk"], case["d"], kv_heads=case["kv_heads"],
                         causal=case["causal"], dtype=case["dtype"])
    if case["kind"] == "forward":
        return llsa.dense_forward(p, st["q"], st["k"], st["v"], q_len=st["q_len"], k_len=st["k_len"])
    return llsa.dense_backward(p, st["q"], st["k"], st["v"], st["o"], st["lse"], st["dout"], q_len=st["q_len"],
                               k_len=st["k_len"])


def run(state):
    return _call(state) if own else _plain(state)


# ------------------------------------------------------- from the definitions

def _exact_turn(case, x, pos, sign):
    """Each pair of columns as a complex number, turned on the unit circle."""
    n, axes = x.shape[2], case["axes"]
    rot = case.get("rot") or case["d"]
    seg = rot // axes
    half = case.get("layout", "half") == "half"
    out = x.double().clone()
    factor, scaling, base = case.get("factor", 1.0), case.get("scaling", "none"), case.get("base", 10000.0)
    amplitude = 0.1 * math.log(factor) + 1.0 if scaling == "wavelength" else 1.0
    for axis in range(axes):
        if pos is not None:
            p = pos[:, :, axis].double()
        else:
            where = []
            for t in range(n):
                if axes == 1:
                    where.append(t + case.get("offset", 0))
                elif case.get("order", "raster") == "raster":
                    where.append(divmod(t, case["width"])[axis])
                else:
                    got, place, rest = 0, 1, t
                    while rest:
                        got += place * ((rest % 16) // 4 if axis == 0 else rest % 4)
                        place, rest = place * 4, rest // 16
                    where.append(got)
            p = torch.tensor(where, dtype=torch.float64, device=x.device)[None]
        for i in range(seg // 2):
            if scaling == "base":
                w = (base * factor ** (seg / (seg - 2.0))) ** (-2.0 * i / seg)
            else:
                w = base ** (-2.0 * i / seg)
            if scaling == "linear":
                w /= factor
            if scaling == "wavelength":
                g = min(1.0, max(0.0, (case["orig_len"] * w / (2 * math.pi) - 1.0) / 31.0))
                w = g * w + (1 - g) * w / factor
            at = axis * seg
            ia, ib = (at + i, at + i + seg // 2) if half else (at + 2 * i, at + 2 * i + 1)
            z = torch.complex(x[..., ia].double(), x[..., ib].double())
            z = z * torch.polar(torch.full_like(p, amplitude), sign * w * p)[:, None]
            out[..., ia], out[..., ib] = z.real, z.imag
    return out


def exact(case, seed):
    kind = case["kind"]
    if kind != "rope" and case["batch"] * case["heads"] * case["nq"] * case["nk"] * case["d"] > 6e10:
        return None  # 64-bit products at that size take too long
    if kind == "rope" and case["batch"] * (case["heads"] + case["kv_heads"]) * case["n"] * case["d"] > 3e8:
        return None
    st = prepare(case, seed)
    if kind == "rope":
        sign = -1.0 if case["inverse"] else 1.0
        return tuple(_exact_turn(case, st[x], st["pos"], sign) for x in "qk")
    q, k, v = (st[x].detach().double() for x in "qkv")
    if kind == "step":
        q, k = (_exact_turn(case, x, None, 1.0) for x in (q, k))
    b, h, kv, nq, nk, d = (case[x] for x in ("batch", "heads", "kv_heads", "nq", "nk", "d"))
    lq, lk = _lengths(case, "q") or [nq] * b, _lengths(case, "k") or [nk] * b
    o, dq = torch.zeros_like(q), torch.zeros_like(q)
    dk, dv = torch.zeros_like(k), torch.zeros_like(v)
    lse = torch.full((b, h, nq), -_INF, dtype=torch.float64, device=q.device)
    for e in range(b):
        a, z = lq[e], lk[e]
        if a == 0 or z == 0:
            continue
        for head in range(h):
            kh = head // (h // kv)
            s = q[e, head, :a] @ k[e, kh, :z].T / math.sqrt(d)
            if case["causal"]:
                s = torch.where(torch.ones_like(s, dtype=torch.bool).tril(z - a), s, -_INF)
            lse[e, head, :a] = torch.logsumexp(s, -1)
            p = torch.where(torch.isinf(lse[e, head, :a])[:, None], torch.zeros_like(s), torch.exp(s - lse[e, head, :a, None]))
            o[e, head, :a] = p @ v[e, kh, :z]
            if kind == "forward":
                continue
            do = st["dout"][e, head, :a].double()
            dp = do @ v[e, kh, :z].T
            ds = p * (dp - (do * o[e, head, :a]).sum(-1, keepdim=True))
            dv[e, kh, :z] += p.T @ do
            dq[e, head, :a] = ds @ k[e, kh, :z] / math.sqrt(d)
            dk[e, kh, :z] += ds.T @ q[e, head, :a] / math.sqrt(d)
    if kind == "forward":
        return o, lse
    if kind == "backward":
        return dq, dk, dv
    dq, dk = (_exact_turn(case, x, None, -1.0) for x in (dq, dk))
    return o, dq, dk, dv
