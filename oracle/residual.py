"""The residual stream's operators in 64 bits: the embedding lookup and its
gradient, dropout from Philox4x32-10, and the joint of a block's output with the
stream.  Test infrastructure; plain definitions on torch CPU tensors.

Each function that a kernel is compared with returns, beside the values, the bar of
every element, derived from the kernels' arithmetic.  With u = 2^-24 (half an fp32
step) and ut half a step of the storage type:

* a sum of terms, each formed with a few roundings, is off by at most
  (depth + a few) u times the sum of the terms' absolute values, depth being the
  longest chain of additions that a term goes through.  Row sums: a thread's own
  columns (at most H / 256 + 32), the warp's five steps and at most 32 warps, taken
  as H / 256 + 72 with the terms' own roundings.  Column sums: at most every row of
  the batch, the CTA's groups and the reduction's steps, taken as T + 72.
* r = rsqrt(mean + eps) carries half of its sum's error and the 2 ulp (4 u) of the
  hardware's reciprocal square root.
"""
from __future__ import annotations

import math

import numpy as np
import torch

U = 2.0 ** -24
TINY = 2.0 ** -126  # below the smallest normal number nothing is relative


def half_step(dtype) -> float:
    return torch.finfo(dtype).eps / 2


def d(t):
    return None if t is None else t.detach().cpu().double()


# ---------------------------------------------------------------- dropout

def philox4x32(counter, key, rounds: int = 10):
    """Philox4x32 (Salmon, Moraes, Dror and Shaw, SC 2011) of four words of
    counter (arrays) and two of key."""
    c = [np.asarray(x, dtype=np.uint64) for x in counter]
    k = [np.uint64(key[0]), np.uint64(key[1])]
    low, half = np.uint64(0xFFFFFFFF), np.uint64(32)
    for _ in range(rounds):
        a, b = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(b >> half) ^ c[1] ^ k[0], b & low, (a >> half) ^ c[3] ^ k[1], a & low]
        k = [(k[0] + np.uint64(0x9E3779B9)) & low, (k[1] + np.uint64(0xBB67AE85)) & low]
    return c


def threshold(p: float) -> int:
    return int(math.floor(65536.0 * p + 0.5))


def keep_mask(T: int, H: int, p: float, seed: int, offset: int = 0, step: int = 0):
    """bool [T, H]."""
    at = (offset + step) % 2 ** 64
    words = philox4x32((np.arange((H + 7) // 8)[None, :], np.arange(T)[:, None],
                        at & 0xFFFFFFFF, at >> 32), (seed & 0xFFFFFFFF, seed >> 32))
    words = np.broadcast_arrays(*words)
    halves = np.stack([h for w in words for h in (w & np.uint64(0xFFFF), w >> np.uint64(16))], -1)
    return torch.from_numpy(halves.reshape(T, -1)[:, :H].astype(np.int64) >= threshold(p))


def drop_scale(p: float) -> float:
    thr = threshold(p)
    return 65536.0 / (65536 - thr) if thr < 65536 else 0.0


def dropout(x, p, seed, offset=0, step=0):
    """(y, bar): the product, its scale and the result rounded once each."""
    keep = keep_mask(*x.shape, p, seed, offset, step)
    y = torch.where(keep, d(x) * drop_scale(p), 0.0)
    return y, (half_step(x.dtype) + 2 * U) * y.abs() + TINY


# -------------------------------------------------------------- embedding

def embed_fwd(W, ids, scale=1.0):
    W64, ids = d(W), ids.cpu().long()
    there = (ids >= 0) & (ids < W.shape[0])
    x = torch.where(there[:, None], W64[ids.clamp(0, W.shape[0] - 1)] * scale, 0.0)
    return x, (half_step(W.dtype) + 2 * U) * x.abs() + TINY


def embed_bwd(dx, ids, V, scale=1.0, base=None):
    """(dW, bar); base: what accumulate adds to."""
    dx64, ids = d(dx), ids.cpu().long()
    there = (ids >= 0) & (ids < V)
    ids, dx64 = ids[there], dx64[there]
    dW = torch.zeros(V, dx.shape[1], dtype=torch.float64)
    mag = torch.zeros_like(dW).index_add_(0, ids, dx64.abs() * abs(scale))
    dW.index_add_(0, ids, dx64 * scale)
    count = torch.bincount(ids, minlength=V).double()[:, None]
    bar = (count + 4) * U * mag
    if base is not None:
        dW += d(base)
        bar += U * dW.abs() * (count > 0)
    return dW, bar + TINY * (count > 0)


# --------------------------------------------------------- a block's joint

def _factors(x, w_post, gate, gate_tok):
    T, H = x.shape
    one = torch.ones
    return (one(H, dtype=torch.float64) if w_post is None else d(w_post),
            one(H, dtype=torch.float64) if gate is None else d(gate),
            one(T, 1, dtype=torch.float64) if gate_tok is None else d(gate_tok).reshape(T, 1))


def rstd_error(H: int) -> float:
    """Relative error of r: half of the sum's, and the reciprocal root's."""
    return ((H / 256 + 72) / 2 + 5) * U


def block_fwd(x, res, w, eps, w_post=None, gate=None, gate_tok=None, res_scale=1.0, x_scale=1.0,
              keep=None, p=0.0):
    """(h, rstd_post) and their bars; rstd_post None without w_post.  The second
    norm is of the stored h: see block_y."""
    T, H = x.shape
    wp, g, gt = _factors(x, w_post, gate, gate_tok)
    x64 = d(x)
    r1 = None
    b = x64 * wp * g * gt
    if w_post is not None:
        r1 = (x64.square().mean(1, keepdim=True) + eps) ** -0.5
        b = b * r1
    if keep is not None:
        b = torch.where(keep, b * drop_scale(p), 0.0)
    b, a = b * x_scale, res_scale * d(res)
    h = a + b
    er = rstd_error(H)
    bar = half_step(x.dtype) * h.abs() + 2 * U * (a.abs() + h.abs()) + (er + 8 * U) * b.abs() + TINY
    return (h, None if r1 is None else r1[:, 0]), (bar, None if r1 is None else er * r1[:, 0])


def block_y(h, w, eps):
    """(y, rstd) of the stored h, and their bars."""
    h64 = d(h)
    r = (h64.square().mean(1, keepdim=True) + eps) ** -0.5
    y, er = h64 * r * d(w), rstd_error(h.shape[1])
    return (y, r[:, 0]), ((half_step(h.dtype) + er + 3 * U) * y.abs() + TINY, er * r[:, 0])


def block_bwd(dy, dh, x, h, w, rstd, rstd_post=None, w_post=None, gate=None, gate_tok=None,
              res_scale=1.0, x_scale=1.0, keep=None, p=0.0):
    """(dx, dres, dw, dw_post, dgate, dgate_tok) and their bars, None where the
    factor is."""
    T, H = x.shape
    ut = half_step(x.dtype)
    wp, g, gt = _factors(x, w_post, gate, gate_tok)
    x64, h64, dy64, dh64, w64, r2 = d(x), d(h), d(dy), d(dh), d(w), d(rstd).reshape(T, 1)
    r1 = torch.ones(T, 1, dtype=torch.float64) if w_post is None else d(rstd_post).reshape(T, 1)
    beta = x_scale * (1.0 if keep is None else drop_scale(p))
    m = torch.ones(T, H, dtype=torch.float64) if keep is None else keep.double()
    es = (H / 256 + 80) * U  # of a row sum, the products of its terms included

    hn, xn, wg = h64 * r2, x64 * r1, wp * g
    wd = w64 * dy64
    k = r2 / H * (wd * hn).sum(1, keepdim=True)
    ek = r2 / H * es * (wd * hn).abs().sum(1, keepdim=True) + 3 * U * k.abs()
    G = dh64 + r2 * wd - k * hn
    eG = ek * hn.abs() + 4 * U * (dh64.abs() + (r2 * wd).abs() + (k * hn).abs())
    q = m * wg * xn
    c = beta * (q * G).sum(1, keepdim=True)
    ec = abs(beta) * (es * (q.abs() * (dh64.abs() + (r2 * wd).abs())).sum(1, keepdim=True)
                      + (ek + es * k.abs()) * (q * hn).abs().sum(1, keepdim=True)) \
        + 4 * U * c.abs()
    dres = res_scale * G
    bres = (ut + U) * dres.abs() + abs(res_scale) * eG + TINY
    one = r1 * beta * gt * m * wg
    two = r1 / H * gt * xn if w_post is not None else torch.zeros_like(xn)
    dx = one * G - two * c
    bx = ut * dx.abs() + one.abs() * (eG + 8 * U * G.abs()) \
        + two.abs() * (ec + 8 * U * c.abs()) + 2 * U * dx.abs() + TINY
    col = (T + 72) * U
    dw = (dy64 * hn).sum(0)
    bw = (col + 2 * U) * (dy64 * hn).abs().sum(0) + TINY
    s = beta * gt * m * xn
    S = (s * G).sum(0)
    bS = (s.abs() * (eG + (col + 6 * U) * G.abs())).sum(0) + TINY

    def shared(factor, there):
        if not there:
            return None, None
        return S * factor, (bS + 3 * U * S.abs()) * factor.abs() + TINY

    dwp, bwp = shared(g, w_post is not None)
    dg, bg = shared(wp, gate is not None)
    dt, bt = (c[:, 0], ec[:, 0] + TINY) if gate_tok is not None else (None, None)
    return (dx, dres, dw, dwp, dg, dt), (bx, bres, bw, bwp, bg, bt)
