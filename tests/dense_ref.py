"""64-bit references of dense attention and rotary positions for the tests, with
error bounds next to the values.

Bounds count roundings. u is half a step of the outputs' type (bf16 2^-8, fp32
2^-24), w that of the type in which the probabilities and dS enter their
products (bf16 for bf16 inputs, else fp32). Sums of m terms in fp32 add at most
m 2^-24 of the sum of magnitudes; `f` covers those (m = d + n terms, and 32 more
for exp, the running rescaling and the joins of a split).

  o   u |o| + (w + f) P|V|                            (P|V| = sum_j P |v_j|)
  lse f max_j |s|_j + n 2^-24 + 4 * 2^-24 |lse| + 2^-20   (|s|_j = scale sum |q||k_j|)
  D   sum |dO| bound(o) + f sum |dO||o|
  dS  (w + f) |dS| + P (bound(D) + f |dP| + f (|dP| + |D|) |s|)
  dv  u |dv| + (w + f + f |s|) P^T |dO|
  dq  u |dq| + scale (bound(dS) + f |dS|) |K|, dk with |Q| the same
A relative error e of P (f |s|: the score's error) stands beside w where it matters.
"""
import math

import torch

INF = float("inf")


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def allowed(nq, nk, lq, lk, causal):
    i, j = torch.arange(nq)[:, None], torch.arange(nk)[None, :]
    ok = (i < lq) & (j < lk)
    return ok & (j <= i + lk - lq) if causal else ok


def attention(q, k, v, dout=None, causal=False, scale=0.0, q_len=None, k_len=None, dtype=torch.bfloat16):
    """{name: (value, bound)} of o, lse and, with dout, dq, dk, dv. Rows and keys
    outside the lengths may hold anything."""
    b, h, nq, d = q.shape
    kv, nk = k.shape[1], k.shape[2]
    scale = scale or 1 / math.sqrt(d)
    u = half_step(dtype)
    w = u
    f = (d + max(nq * h // kv, nk) + 32) * 2.0 ** -24
    out = {n: (torch.zeros(s, dtype=torch.float64), torch.zeros(s, dtype=torch.float64)) for n, s in
           (("o", q.shape), ("dq", q.shape), ("dk", k.shape), ("dv", k.shape))}
    out["lse"] = (torch.full((b, h, nq), -INF, dtype=torch.float64), torch.zeros(b, h, nq, dtype=torch.float64))
    for e in range(b):
        lq = nq if q_len is None else int(q_len[e])
        lk = nk if k_len is None else int(k_len[e])
        if lq == 0 or lk == 0:
            continue
        ok = allowed(lq, lk, lq, lk, causal)
        for hh in range(h):
            g = hh // (h // kv)
            Q, K, V = q[e, hh, :lq].double(), k[e, g, :lk].double(), v[e, g, :lk].double()
            s = (scale * Q @ K.T).masked_fill(~ok, -INF)
            mag = (scale * Q.abs() @ K.abs().T).masked_fill(~ok, 0.0)
            lse = torch.logsumexp(s, -1)
            P = torch.exp(s - lse.masked_fill(lse == -INF, 0.0)[:, None])
            o = P @ V
            rel = f * (1 + mag)  # relative error of a probability
            o_err = u * o.abs() + ((w + rel) * P) @ V.abs() + f * o.abs()
            out["o"][0][e, hh, :lq], out["o"][1][e, hh, :lq] = o, o_err
            out["lse"][0][e, hh, :lq] = lse
            out["lse"][1][e, hh, :lq] = f * mag.amax(-1) + lk * 2.0 ** -24 + 4 * 2.0 ** -24 * lse.abs().nan_to_num(posinf=0) + 2.0 ** -20
            if dout is None:
                continue
            G = dout[e, hh, :lq].double()
            D = (G * o).sum(-1, keepdim=True)
            dP = G @ V.T
            dP_mag = G.abs() @ V.abs().T
            D_err = (G.abs() * o_err).sum(-1, keepdim=True) + f * (G.abs() * o.abs()).sum(-1, keepdim=True)
            dS = P * (dP - D)
            # the lse that comes in carries its own error: another relative error of P
            rel = rel + out["lse"][1][e, hh, :lq][:, None]
            dS_err = (w + f) * dS.abs() + P * (D_err + f * dP_mag + rel * (dP.abs() + D.abs()))
            dv_err = ((w + rel) * P).T @ G.abs()
            out["dq"][0][e, hh, :lq] = scale * dS @ K
            out["dq"][1][e, hh, :lq] = u * (scale * dS @ K).abs() + scale * (dS_err + f * dS.abs()) @ K.abs()
            out["dk"][0][e, g, :lk] += scale * dS.T @ Q
            out["dk"][1][e, g, :lk] += scale * (dS_err + f * dS.abs()).T @ Q.abs()
            out["dv"][0][e, g, :lk] += P.T @ G
            out["dv"][1][e, g, :lk] += dv_err + f * (P.T @ G.abs())
    for n in ("dk", "dv"):  # rounded once, after the sum over the heads that share the key head
        out[n][1].add_(u * out[n][0].abs())
    return out


def check(name, got, ref):
    """got within the bound of ref = (value, bound), element by element; infinities equal."""
    value, bound = ref
    got = got.detach().double().cpu()
    assert got.shape == value.shape, (name, got.shape, value.shape)
    fine = torch.isfinite(value)
    assert torch.equal(got[~fine], value[~fine]), f"{name}: infinities differ"
    err = (got - value).abs()[fine]
    over = err > bound[fine] + 1e-30
    assert not bool(over.any()) and not bool(err.isnan().any()), (
        f"{name}: {int(over.sum())} of {err.numel()} values off, worst {float(err.max()):.3e}, "
        f"largest excess {float((err - bound[fine]).max()):.3e}")


# ------------------------------------------------------------------- rotary

def frequencies(seg, base=10000.0, scaling="none", factor=1.0, orig_len=0, low=1.0, high=32.0):
    got = []
    for i in range(seg // 2):
        b = base * factor ** (seg / (seg - 2)) if scaling == "base" else base
        w = b ** (-2.0 * i / seg)
        if scaling == "linear":
            w /= factor
        if scaling == "wavelength":
            g = min(1.0, max(0.0, (orig_len * w / (2 * math.pi) - low) / (high - low)))
            w *= g + (1 - g) / factor
        got.append(w)
    return got


def rotary(x, pos, rot=0, layout="half", axes=1, inverse=False, amplitude=0.0, dtype=None, **kw):
    """(value, bound) of x [batch, heads, n, d] turned by pos [1 or batch, n, axes]."""
    d = x.shape[-1]
    rot = rot or d
    seg = rot // axes
    A = amplitude or (0.1 * math.log(kw["factor"]) + 1 if kw.get("scaling") == "wavelength" else 1.0)
    x = x.double()
    out, bound = x.clone(), torch.zeros_like(x)
    u = half_step(dtype) if dtype is not None else 0.0
    for a in range(axes):
        for i, w in enumerate(frequencies(seg, **kw)):
            p = pos[..., a].double()
            ang = (-p if inverse else p) * w
            c, s = (A * ang.cos())[:, None], (A * ang.sin())[:, None]
            ia, ib = (a * seg + i, a * seg + i + seg // 2) if layout == "half" else (a * seg + 2 * i, a * seg + 2 * i + 1)
            X, Y = x[..., ia], x[..., ib]
            out[..., ia], out[..., ib] = X * c - Y * s, X * s + Y * c
            # cos and sin are good to 2^-22; w carries roundings of 2^-52 that the position multiplies
            bound[..., ia] = bound[..., ib] = A * (X.abs() + Y.abs()) * (2.0 ** -21 + 2.0 ** -50 * p.abs()[:, None])
    bound[..., :rot] += u * out[..., :rot].abs()
    return out, bound
