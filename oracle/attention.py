"""Attention over packed sequences and the multi-axis rotation in double
precision, with the error bars their tests use (test infrastructure only).

Plain torch in float64, one (sequence, head) at a time, on whatever device the
inputs are.  Bars are first-order bounds by arithmetic, with u = 2^-24 (fp32,
half a step), r = 2^-8 for bf16 storage or u for fp32 storage (the rounding of
an output, and of the probabilities and score gradients that enter a second
product; fp32 storage keeps those in fp32), and a sum of n terms in fp32 off by
at most (n + 3) 2u times the sum of the terms' magnitudes, where 2u instead of u allows
for an accumulator that truncates:

  E_s = (D + 3) 2u |scale| sum_d |q k|          error of one score
  a row's exponent: the score's error, that of the maximum it is taken from and
  the exponential's own: 2 max_j E_s + X, X = (8 + 3 |s - lse|_max) u
"""
import math

import torch

U = 2.0 ** -24
R = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}


def _sequences(cu):
    c = [int(x) for x in cu]
    return [(a, b) for a, b in zip(c[:-1], c[1:]) if b > a]


def _scores(q, k, scale, causal):
    z = scale * (q @ k.T)
    mag = abs(scale) * (q.abs() @ k.abs().T)
    if causal:
        hidden = torch.ones_like(z, dtype=torch.bool).triu(1)
        z = z.masked_fill(hidden, -math.inf)
        mag = mag.masked_fill(hidden, 0.0)
    return z, mag


def attn_fwd(q, k, v, cu, scale, causal, code):
    """(o, lse, bar of o, bar of lse); rows of no sequence hold NaN."""
    q, k, v = q.double(), k.double(), v.double()
    T, Hq, D = q.shape
    G = Hq // k.shape[1]
    o, ob = torch.full_like(q, math.nan), torch.full_like(q, math.nan)
    lse = torch.full((Hq, T), math.nan, dtype=torch.float64, device=q.device)
    lb = lse.clone()
    for a, b in _sequences(cu):
        for h in range(Hq):
            qs, ks, vs = q[a:b, h], k[a:b, h // G], v[a:b, h // G]
            z, mag = _scores(qs, ks, scale, causal)
            norm = torch.logsumexp(z, 1)
            p = torch.exp(z - norm[:, None])
            es = (D + 3) * 2 * U * mag.amax(1) + U * z.amax(1).abs()
            far = (norm[:, None] - z).masked_fill(p == 0, 0.0).amax(1)
            e = 2 * es + (8 + 3 * far) * U + (b - a + 3) * 2 * U
            r = p @ vs
            rmag = p @ vs.abs()
            o[a:b, h] = r
            # the probabilities' rounding, every fp32 step of p, l and p v, the store
            ob[a:b, h] = (R[code] + 2 * e[:, None] + (b - a + 3) * 2 * U) * rmag + R[code] * r.abs()
            lse[h, a:b] = norm
            lb[h, a:b] = e + 4 * U * (norm.abs() + math.log(b - a + 1))
    return o, lse, ob, lb


def attn_bwd(do, q, k, v, o, lse, cu, scale, causal, code):
    """((dq, dk, dv), their bars) from the given o and lse."""
    do, q, k, v, o, lse = (x.double() for x in (do, q, k, v, o, lse))
    T, Hq, D = q.shape
    G = Hq // k.shape[1]
    out = [torch.full_like(x, math.nan) for x in (q, k, v)]
    bar = [torch.full_like(x, math.nan) for x in (q, k, v)]
    dq, dk, dv = out
    bq, bk, bv = bar
    r = R[code]
    for a, b in _sequences(cu):
        n = b - a
        for x in (dk, dv, bk, bv):
            x[a:b] = 0.0
        for h in range(Hq):
            hk = h // G
            qs, ks, vs, gs, os_ = q[a:b, h], k[a:b, hk], v[a:b, hk], do[a:b, h], o[a:b, h]
            z, mag = _scores(qs, ks, scale, causal)
            p = torch.exp(z - lse[h, a:b, None])
            far = (lse[h, a:b, None] - z).abs().masked_fill(torch.isinf(z), 0.0)
            # relative error of p: the score's, the exponent's steps, the exponential's
            ep = (D + 3) * 2 * U * mag + (8 + 3 * far + 2 * lse[h, a:b, None].abs()) * U
            delta = (gs * os_).sum(1, keepdim=True)
            dp = gs @ vs.T
            ds = p * (dp - delta)
            eds = ds.abs() * (ep + 4 * U) + p * (D + 3) * 2 * U * (
                gs.abs() @ vs.abs().T + (gs * os_).abs().sum(1, keepdim=True))
            m = ds.abs() * r + eds  # what a score gradient may be off by, rounding included
            acc = (G * n + 3) * 2 * U
            dq[a:b, h] = scale * (ds @ ks)
            bq[a:b, h] = scale * ((m + acc * ds.abs()) @ ks.abs()) + r * dq[a:b, h].abs()
            dk[a:b, hk] += scale * (ds.T @ qs)
            bk[a:b, hk] += scale * ((m + acc * ds.abs()).T @ qs.abs())
            dv[a:b, hk] += p.T @ gs
            bv[a:b, hk] += (p * (r + ep + acc)).T @ gs.abs()
        bk[a:b] += r * dk[a:b].abs()
        bv[a:b] += r * dv[a:b].abs()
    return out, bar


def qk_mrope(x, pos, axis_of, inv_freq, sign, code):
    """(y, bar) of one of q, k [T, H, D]; inv_freq: D/2 doubles."""
    x = x.double()
    half = x.shape[2] // 2
    f = torch.as_tensor(inv_freq, dtype=torch.float64, device=x.device)
    axis = torch.as_tensor(axis_of, device=x.device).long()
    phi = sign * pos.double()[axis].T * f
    c, s = phi.cos()[:, None], phi.sin()[:, None]
    a, b = x[..., :half], x[..., half:]
    y = torch.cat([a * c - b * s, b * c + a * s], -1)
    mag = torch.cat([(a * c).abs() + (b * s).abs(), (b * c).abs() + (a * s).abs()], -1)
    turn = torch.cat([(a * s).abs() + (b * c).abs(), (b * s).abs() + (a * c).abs()], -1)
    # three fp32 roundings of each term, the cosine's own error (4u) and an
    # angle off by 1e-6 rad below position 2^20 (by 2^-46 of the turns beyond)
    angle = 1e-6 + pos.double().abs().amax() * 2.0 ** -46
    return y, 8 * U * mag + (angle + 4 * U) * turn + R[code] * y.abs() + 2.0 ** -126
