"""64-bit reference of differential attention for the tests, with error bounds next to
the values; the notation and the counting of roundings are those of dense_ref.

With a^i = P^i V, w_1 = 1, w_2 = -lam, e(a^i) = (w + f (1 + |s|)) P^i|V| + f |a^i|:
  o2   u |o2| + e(a^2)
  o    u |o| + e(a^1) + |lam| e(a^2) + f (|a^1| + |lam| |a^2|)
  D^2  sum |dO| bound(o2) + f sum |dO||o2|
  D^1  it comes from o + lam o2: sum |dO| (bound(o) + |lam| bound(o2)) + f sum |dO| (|o| + 2 |lam| |o2|)
  dS^i |w_i| ((w + f) P|dP - D| + P (bound(D^i) + f |dP| + rel (|dP| + |D|))), rel = f (1 + |s|) + bound(lse)
  dv   u |dv| + sum_i |w_i| (w + rel) P^i^T |dO|   (rounded together or apart, a weight's rounding is at most w of P^1 + |lam| P^2)
  dq, dk: as dense_ref
  dlam u |dlam| + sum |dO| bound(o2) + g sum |dO||o2|, g = 2^-24 times the longest chain of additions
"""
import math

import torch

from dense_ref import INF, allowed, check, half_step  # noqa: F401


def attention(q, k, v, lam, dout=None, causal=False, scale=0.0, q_len=None, k_len=None, dtype=torch.bfloat16, lam_dtype=None):
    """{name: (value, bound)} of o, o2, lse and, with dout, dq, dk, dv, dlam."""
    b, h2, nq, d = q.shape
    h, kv, nk = h2 // 2, v.shape[1], k.shape[2]
    scale = scale or 1 / math.sqrt(d)
    u = w = half_step(dtype)
    f = (2 * d + max(nq * h // kv, nk) + 32) * 2.0 ** -24
    z = lambda *s: torch.zeros(*s, dtype=torch.float64)
    out = {n: (z(s), z(s)) for n, s in (("o", (b, h, nq, 2 * d)), ("o2", (b, h, nq, 2 * d)), ("dq", q.shape), ("dk", k.shape),
                                        ("dv", v.shape), ("dlam", (h,)))}
    out["lse"] = (torch.full((b, h2, nq), -INF, dtype=torch.float64), z(b, h2, nq))
    chain = (b * nq * 2 * d / 256 + 700) * 2.0 ** -24
    for e in range(b):
        lq = nq if q_len is None else int(q_len[e])
        lk = nk if k_len is None else int(k_len[e])
        if lq == 0 or lk == 0:
            continue
        ok = allowed(lq, lk, lq, lk, causal)
        for hh in range(h):
            g = hh // (h // kv)
            L = float(lam[hh])
            V = v[e, g, :lk].double()
            maps = []
            for i in (0, 1):
                Q, K = q[e, i * h + hh, :lq].double(), k[e, i * kv + g, :lk].double()
                s = (scale * Q @ K.T).masked_fill(~ok, -INF)
                mag = (scale * Q.abs() @ K.abs().T).masked_fill(~ok, 0.0)
                lse = torch.logsumexp(s, -1)
                P = torch.exp(s - lse.masked_fill(lse == -INF, 0.0)[:, None])
                A, rel = P @ V, f * (1 + mag)
                A_err = ((w + rel) * P) @ V.abs() + f * A.abs()
                l_err = f * mag.amax(-1) + lk * 2.0 ** -24 + 4 * 2.0 ** -24 * lse.abs().nan_to_num(posinf=0) + 2.0 ** -20
                out["lse"][0][e, i * h + hh, :lq], out["lse"][1][e, i * h + hh, :lq] = lse, l_err
                maps.append((Q, K, P, A, A_err, rel, l_err))
            A, B = maps[0][3], maps[1][3]
            o, o_err = A - L * B, maps[0][4] + abs(L) * maps[1][4] + f * (A.abs() + abs(L) * B.abs())
            o_err = o_err + u * o.abs()
            b_err = maps[1][4] + u * B.abs()
            out["o"][0][e, hh, :lq], out["o"][1][e, hh, :lq] = o, o_err
            out["o2"][0][e, hh, :lq], out["o2"][1][e, hh, :lq] = B, b_err
            if dout is None:
                continue
            G = dout[e, hh, :lq].double()
            ga = G.abs()
            live = ok.any(-1, keepdim=True)
            dP, dP_mag = G @ V.T, ga @ V.abs().T
            D_errs = ((ga * (o_err + abs(L) * b_err)).sum(-1, keepdim=True) + f * (ga * (o.abs() + 2 * abs(L) * B.abs())).sum(-1, keepdim=True),
                      (ga * b_err).sum(-1, keepdim=True) + f * (ga * B.abs()).sum(-1, keepdim=True))
            out["dlam"][0][hh] -= (G * B * live).sum()
            out["dlam"][1][hh] += (ga * b_err * live).sum() + chain * (ga * B.abs() * live).sum()
            for i, (Q, K, P, Ai, _, rel, l_err) in enumerate(maps):
                wi = 1.0 if i == 0 else -L
                D = (G * Ai).sum(-1, keepdim=True)
                rel = rel + l_err.nan_to_num(posinf=0)[:, None]
                dS = wi * P * (dP - D)
                dS_err = (w + f) * dS.abs() + abs(wi) * P * (D_errs[i] + f * dP_mag + rel * (dP.abs() + D.abs()))
                out["dq"][0][e, i * h + hh, :lq] = scale * dS @ K
                out["dq"][1][e, i * h + hh, :lq] = u * (scale * dS @ K).abs() + scale * (dS_err + f * dS.abs()) @ K.abs()
                out["dk"][0][e, i * kv + g, :lk] += scale * dS.T @ Q
                out["dk"][1][e, i * kv + g, :lk] += scale * (dS_err + f * dS.abs()).T @ Q.abs()
                out["dv"][0][e, g, :lk] += wi * P.T @ G
                out["dv"][1][e, g, :lk] += abs(wi) * (((w + rel) * P).T @ ga + f * (P.T @ ga))
    for n in ("dk", "dv", "dlam"):  # rounded once, after the sum over the heads that share the key head
        ul = half_step(lam_dtype or dtype) if n == "dlam" else u
        out[n][1].add_(ul * out[n][0].abs())
    return out


def lam_gradient(q, k, v, lam, dout, causal=False, scale=0.0, q_len=None, k_len=None, lam_dtype=torch.float32):
    """(value, bound) of dlam where it is summed from P_2 dP in fp32, as the kernels for bf16 do.
    A pair's term is off by the score's sums of d exact products, (d + 32) 2^-24 of their magnitude, by the
    exponential, 2^-22, and its argument, 2^-23 of ln P, and by dP's sums of 2 d, (2 d + 32) 2^-24 of theirs; all
    pairs of a row alike by lse and its product with log2 e, which so stands beside the row's D_2; and the
    terms are added in chains of at most nk + rows + 700. Nothing is rounded to bf16 but the result to lam's type."""
    b, h2, nq, d = q.shape
    h, kv, nk = h2 // 2, v.shape[1], k.shape[2]
    scale = scale or 1 / math.sqrt(d)
    e24 = 2.0 ** -24
    f = (2 * d + max(nq * h // kv, nk) + 32) * e24
    value, bound = torch.zeros(h, dtype=torch.float64), torch.zeros(h, dtype=torch.float64)
    for e in range(b):
        lq = nq if q_len is None else int(q_len[e])
        lk = nk if k_len is None else int(k_len[e])
        if lq == 0 or lk == 0:
            continue
        ok = allowed(lq, lk, lq, lk, causal)
        for hh in range(h):
            g = hh // (h // kv)
            Q, K, V = q[e, h + hh, :lq].double(), k[e, kv + g, :lk].double(), v[e, g, :lk].double()
            G = dout[e, hh, :lq].double()
            s = (scale * Q @ K.T).masked_fill(~ok, -INF)
            mag = (scale * Q.abs() @ K.abs().T).masked_fill(~ok, 0.0)
            lse = torch.logsumexp(s, -1)
            live = lse > -INF
            ln = s - lse.masked_fill(~live, 0.0)[:, None]
            P, dP = torch.exp(ln), G @ V.T
            D = (P * dP).sum(-1)
            l_err = f * mag.amax(-1) + lk * e24 + 6 * e24 * lse.abs().nan_to_num(posinf=0) + 2.0 ** -20
            rel = (d + 32) * e24 * (1 + mag) + 2.0 ** -22 + 2 * e24 * ln.abs().nan_to_num(posinf=0)
            value[hh] -= D[live].sum()
            bound[hh] += (l_err * D.abs())[live].sum() + (P * (rel * dP.abs() + (2 * d + 32) * e24 * (G.abs() @ V.abs().T))).sum()
            bound[hh] += (nk + b * nq + 700) * e24 * (P * dP.abs()).sum()
    return value, bound + half_step(lam_dtype) * value.abs()
