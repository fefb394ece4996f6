"""Measured cases of the packed-sequence attention block: the rotation of Q and
K by positions on several axes, and attention over variable-length packed
sequences with its backward pass.

``run`` computes an operator in plain torch (``own`` false) or through the
library's calls (``own`` true), on the same state; ``exact`` restates the
definitions in 64 bits.  Shapes are those of ``fine_tuning_gb300.workloads``
(head counts, head sizes, length distributions) or generic ones.

Definitions, for sequence b (tokens cu[b] .. cu[b+1]) and query head h, whose
key head is h // (Hq / Hkv):

    s[i, j] = scale * q[i, h] . k[j, h'],   j <= i when causal
    lse[h, i] = log sum_j e^s[i, j],  p = e^(s - lse),  o[i, h] = sum_j p v[j, h']
    dv = p^T do,  dp = do v^T,  ds = p (dp - sum_d do o),
    dq = scale ds k,  dk = scale ds^T q      (dk, dv summed over a group's heads)

    phi_i(t) = pos[axis(i), t] theta^(-2i/D);  the pair (x[i], x[i + D/2]) of
    every head of q and k turns by phi_i (backward: by -phi_i)
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
PIECE = 1 << 31  # score elements that the plain form holds at a time
EXACT_FLOPS = 8e12  # the 64-bit form is left out beyond this


# ------------------------------------------------------------------ lengths

def _lengths(kind, T, seed):
    """Sequence lengths of a packed batch of T tokens."""
    if kind == "one":
        return [T]
    if kind == "tiny":
        return [5, 17, 32, 10]
    rng = np.random.default_rng(seed)
    out, total = [], 0
    while total < T:
        if kind == "lognormal":
            n = int(np.clip(np.rint(rng.lognormal(5.0, 1.0)), 16, 2048))
        elif kind == "half":
            n = int(rng.integers(16, 257)) if rng.random() < 0.5 else int(rng.integers(1024, 4097))
        elif kind == "mix":
            n = int(rng.integers(16, 257)) if rng.random() < 0.8 else int(rng.integers(2048, 8193))
        elif kind == "short":
            n = int(rng.integers(1, 65))
        else:  # "grid": the patches of images of many sizes
            n = int(rng.integers(8, 49)) * int(rng.integers(8, 49))
        n = min(n, T - total)
        out.append(n)
        total += n
    return out


def _pairs(case):
    """Score entries that the mask leaves, over one head."""
    L = _lengths(case["lens"], case["T"], case["len_seed"])
    return sum(n * (n + 1) // 2 if case["causal"] else n * n for n in L)


# ------------------------------------------------------------------ cases

def _attn(name, op, dtype, Hq, Hkv, D, lens, T, len_seed, causal=True, fused=True):
    case = {"op": op, "dtype": dtype, "Hq": Hq, "Hkv": Hkv, "D": D, "lens": lens, "T": T,
            "len_seed": len_seed, "causal": causal, "fused": fused}
    return {"name": name, **case} if name else case


def _rope(name, op, dtype, Hq, Hkv, D, T, theta, fused=True):
    case = {"op": op, "dtype": dtype, "Hq": Hq, "Hkv": Hkv, "D": D, "T": T, "theta": theta,
            "fused": fused}
    return {"name": name, **case} if name else case


def listed():
    return [
        # the fp32 workload of four short sequences: what a call costs at least
        _attn("attn-fwd-tiny-f32", "attn_fwd", "f32", 4, 2, 16, "tiny", 64, 0),
        # Qwen2.5-0.5B heads over a packed instruction-tuning batch: many short sequences, an
        # odd number of query heads for each key head
        _attn("attn-fwd-14x2x64-lognormal", "attn_fwd", "bf16", 14, 2, 64, "lognormal", 16384, 1),
        # Qwen3-8B heads over a batch that mixes chat turns with long documents
        _attn("attn-fwd-32x8x128-mix", "attn_fwd", "bf16", 32, 8, 128, "mix", 32768, 3),
        # Qwen3-32B heads over one long document: the largest
        _attn("attn-fwd-64x8x128-one", "attn_fwd", "bf16", 64, 8, 128, "one", 32768, 4),
        # an image encoder's layer: every patch sees its whole image, a head size that is not a
        # power of two, separate q, k and v
        _attn("attn-fwd-16x16x80-grid", "attn_fwd", "bf16", 16, 16, 80, "grid", 8191, 5,
              causal=False, fused=False),
        _attn("attn-bwd-tiny-f32", "attn_bwd", "f32", 4, 2, 16, "tiny", 64, 0),
        _attn("attn-bwd-14x2x64-lognormal", "attn_bwd", "bf16", 14, 2, 64, "lognormal", 16384, 1),
        # Llama-3.2-1B heads, half the sequences long
        _attn("attn-bwd-32x8x64-half", "attn_bwd", "bf16", 32, 8, 64, "half", 32768, 2),
        # Qwen3-8B heads over one long document
        _attn("attn-bwd-32x8x128-one", "attn_bwd", "bf16", 32, 8, 128, "one", 16384, 3),
        # the rotation of one short prompt with an image
        _rope("mrope-fwd-14x2x64-short", "mrope_fwd", "bf16", 14, 2, 64, 333, 1e6),
        # Qwen3-8B heads over a packed batch of text and video, forward and backward
        _rope("mrope-fwd-32x8x128", "mrope_fwd", "bf16", 32, 8, 128, 65536, 1e6),
        _rope("mrope-bwd-32x8x64-f32", "mrope_bwd", "f32", 32, 8, 64, 32767, 5e5, fused=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attn_fwd", "attn_bwd", "attn_fwd", "attn_bwd", "mrope_fwd", "mrope_bwd"])
    Hkv = rng.choice([1, 2, 3, 4, 8])
    Hq = Hkv * rng.choice([1, 2, 3, 4, 5, 7, 8])
    fused = rng.random() < 0.5
    if op.startswith("mrope"):
        D = rng.choice([16, 32, 64, 80, 96, 128, 256])
        T = _log(rng, 1, max(2, (1 << 27) // ((Hq + Hkv) * D)))
        return _rope("", op, rng.choice(["bf16", "bf16", "f32"]), Hq, Hkv, D, T,
                     rng.choice([1e4, 5e5, 1e6]), fused)
    small = rng.random() < 0.25
    D = rng.choice([16, 33, 48, 64, 128, 160]) if small else rng.choice([64, 64, 72, 80, 96, 128, 128])
    lens = rng.choice(["one", "short", "lognormal", "half", "mix", "grid"])
    most = 2048 if small else 12288 if lens == "one" else 24576
    T = _log(rng, 1, most)
    return _attn("", op, rng.choice(["bf16", "f32"]) if small else "bf16", Hq, Hkv, D, lens, T,
                 rng.randrange(1000), causal=rng.random() < 0.75, fused=fused)


# ------------------------------------------------------------------ inputs

def _normal(gen, shape, dtype, std=1.0):
    t = torch.empty(shape, dtype=torch.float32, device=DEV)
    t.normal_(0.0, std, generator=gen)
    return t.to(dtype)


def _positions(rng, T):
    """Positions [3, T] (time, height, width) of alternating text and video
    spans: a text token moves all three axes by one; a video's frame moves
    time, and its patches' rows and columns the others, from where the text
    stopped; the next text starts past the largest of them."""
    out, at, total = [], 0, 0
    while total < T:
        n = int(rng.integers(1, 400))
        out.append(np.broadcast_to(at + np.arange(n), (3, n)))
        at += n
        total += n
        f, h, w = int(rng.integers(1, 9)), int(rng.integers(2, 25)), int(rng.integers(2, 25))
        t, y, x = np.meshgrid(np.arange(f), np.arange(h), np.arange(w), indexing="ij")
        out.append(at + np.stack([t.ravel(), y.ravel(), x.ravel()]))
        at += max(f, h, w)
        total += f * h * w
    return np.ascontiguousarray(np.concatenate(out, axis=1)[:, :T]).astype(np.int32)


def _axis_of(D):
    """The axis of each of D/2 frequencies, in three runs: a quarter for time,
    and the rest halved between height and width."""
    half = D // 2
    t = half // 4
    h = t + (half - t) // 2
    return np.repeat(np.arange(3), [t, h - t, half - h]).astype(np.int32)


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(int(seed) * 7919 + 17)
    T, Hq, Hkv, D, dtype = case["T"], case["Hq"], case["Hkv"], case["D"], TYPES[case["dtype"]]
    s = {"case": dict(case)}
    if case["fused"]:  # q, k and v as they leave one projection
        qkv = _normal(gen, (T, Hq + 2 * Hkv, D), dtype)
        s["q"], s["k"], s["v"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    else:
        s["q"] = _normal(gen, (T, Hq, D), dtype)
        s["k"], s["v"] = _normal(gen, (T, Hkv, D), dtype), _normal(gen, (T, Hkv, D), dtype)
    if case["op"].startswith("mrope"):
        rng = np.random.default_rng(int(seed) + 1)
        s["pos"] = torch.from_numpy(_positions(rng, T)).to(DEV)
        s["axis_of"], s["theta"] = _axis_of(D), float(case["theta"])
        s["axis"] = torch.from_numpy(s["axis_of"]).to(DEV).long()  # the plain form's index
        return s
    s["lens"] = _lengths(case["lens"], T, case["len_seed"])
    cu = np.concatenate([[0], np.cumsum(s["lens"])]).astype(np.int32)
    s["cu"] = torch.from_numpy(cu).to(DEV)
    s["scale"], s["causal"] = 1.0 / math.sqrt(D), bool(case["causal"])
    if case["op"] == "attn_bwd":  # what the forward pass left, and the gradient that arrives
        s["o"], s["lse"] = _attn_fwd(s)
        s["do"] = _normal(gen, (T, Hq, D), dtype)
    return s


# ------------------------------------------------------------------ plain forms

def _pieces(s):
    """(tokens, key heads) slices whose scores fit in memory together."""
    Hq, Hkv = s["q"].shape[1], s["k"].shape[1]
    G, a = Hq // Hkv, 0
    for n in s["lens"]:
        most = max(1, PIECE // max(1, G * n * n))
        for h in range(0, Hkv, most):
            e = min(Hkv, h + most)
            yield slice(a, a + n), slice(h, e), slice(h * G, e * G)
        a += n


def _by_key_head(x, Hkv):
    """[n, heads, D] -> fp32 [Hkv, heads / Hkv, n, D]."""
    n, H, D = x.shape
    return x.float().reshape(n, Hkv, H // Hkv, D).permute(1, 2, 0, 3)


def _scores(s, q, k):
    z = (q.reshape(k.shape[0], -1, q.shape[-1]) @ k[:, 0].transpose(1, 2)).reshape(
        *q.shape[:3], k.shape[2]) * s["scale"]
    if s["causal"]:
        i = torch.arange(z.shape[-1], device=z.device)
        z.masked_fill_(i[None, :] > i[:, None], -math.inf)
    return z


def _attn_fwd(s):
    q, k, v = s["q"], s["k"], s["v"]
    o = torch.empty(q.shape, dtype=q.dtype, device=q.device)
    lse = torch.empty((q.shape[1], q.shape[0]), dtype=torch.float32, device=q.device)
    for t, hk, hq in _pieces(s):
        Hk = hk.stop - hk.start
        qp, kp, vp = (_by_key_head(x, Hk) for x in (q[t, hq], k[t, hk], v[t, hk]))
        z = _scores(s, qp, kp)
        m = z.amax(-1, keepdim=True)
        p = (z - m).exp_()
        del z
        l = p.sum(-1, keepdim=True)
        r = (p.reshape(Hk, -1, p.shape[-1]) @ vp[:, 0]).reshape(qp.shape) / l
        o[t, hq] = r.permute(2, 0, 1, 3).reshape(r.shape[2], -1, r.shape[3]).to(o.dtype)
        lse[hq, t] = (m + l.log()).reshape(-1, m.shape[2])
    return o, lse


def _attn_bwd(s):
    q, k, v, o, lse, do = (s[n] for n in ("q", "k", "v", "o", "lse", "do"))
    dq, dk, dv = (torch.empty(x.shape, dtype=x.dtype, device=x.device) for x in (q, k, v))
    for t, hk, hq in _pieces(s):
        Hk = hk.stop - hk.start
        qp, op, gp = (_by_key_head(x[t, hq], Hk) for x in (q, o, do))
        kp, vp = (_by_key_head(x[t, hk], Hk) for x in (k, v))
        n = qp.shape[2]
        p = (_scores(s, qp, kp) - lse[hq, t].reshape(Hk, -1, n, 1)).exp_()
        flat = lambda x: x.reshape(Hk, -1, x.shape[-1])  # noqa: E731
        delta = (gp * op).sum(-1, keepdim=True)
        dv[t, hk] = (flat(p).transpose(1, 2) @ flat(gp)).permute(1, 0, 2).to(dv.dtype)
        ds = (flat(gp) @ vp[:, 0].transpose(1, 2)).reshape(p.shape).sub_(delta).mul_(p)
        del p
        ds.mul_(s["scale"])
        g = (flat(ds) @ kp[:, 0]).reshape(qp.shape)
        dq[t, hq] = g.permute(2, 0, 1, 3).reshape(n, -1, g.shape[3]).to(dq.dtype)
        dk[t, hk] = (flat(ds).transpose(1, 2) @ flat(qp)).permute(1, 0, 2).to(dk.dtype)
    return dq, dk, dv


def _mrope(s, sign):
    q, k = s["q"], s["k"]
    half = q.shape[2] // 2
    i = torch.arange(half, dtype=torch.float64, device=q.device)
    phi = s["pos"][s["axis"]].T.double() * s["theta"] ** (-i / half)  # far positions need 64 bits
    c, n = phi.cos().float()[:, None], (sign * phi.sin()).float()[:, None]

    def turn(x):
        a, b = x[..., :half].float(), x[..., half:].float()
        return torch.cat([a * c - b * n, b * c + a * n], -1).to(x.dtype)

    return turn(q), turn(k)


def run(s):
    op = s["case"]["op"]
    if own:
        from fine_tuning_gb300 import ftk
        if op == "attn_fwd":
            return ftk.attn_fwd(s["q"], s["k"], s["v"], s["cu"], scale=s["scale"],
                                causal=s["causal"])
        if op == "attn_bwd":
            return ftk.attn_bwd(s["do"], s["q"], s["k"], s["v"], s["o"], s["lse"], s["cu"],
                                scale=s["scale"], causal=s["causal"])
        turn = ftk.qk_mrope_fwd if op == "mrope_fwd" else ftk.qk_mrope_bwd
        return turn(s["q"], s["k"], s["pos"], s["axis_of"], theta=s["theta"])
    if op == "attn_fwd":
        return _attn_fwd(s)
    if op == "attn_bwd":
        return _attn_bwd(s)
    return _mrope(s, 1.0 if op == "mrope_fwd" else -1.0)


# ------------------------------------------------------------------ cost, definition

def work(case):
    """Bytes: each input read and each output written once.  Operations: the
    products over the score entries that the mask leaves (two forward; five
    backward, with the scores made again), or six for each rotated pair."""
    T, Hq, Hkv, D = case["T"], case["Hq"], case["Hkv"], case["D"]
    es = 2 if case["dtype"] == "bf16" else 4
    qb, kb = T * Hq * D * es, T * Hkv * D * es
    if case["op"].startswith("mrope"):
        return {"bytes": 2 * (qb + kb) + 12 * T, "flops": 3 * T * (Hq + Hkv) * D}
    mul = 2 * _pairs(case) * Hq * D
    if case["op"] == "attn_fwd":
        return {"bytes": 2 * qb + 2 * kb + 4 * T * Hq, "flops": 2 * mul}
    return {"bytes": 4 * qb + 4 * kb + 4 * T * Hq, "flops": 5 * mul}


def exact(case, seed):
    s = prepare(case, seed)
    q, k, v = (s[n].double() for n in ("q", "k", "v"))
    D, G = q.shape[2], q.shape[1] // k.shape[1]
    if case["op"].startswith("mrope"):
        sign = 1.0 if case["op"] == "mrope_fwd" else -1.0
        freq = torch.tensor([case["theta"] ** (-2.0 * i / D) for i in range(D // 2)],
                            dtype=torch.float64, device=DEV)
        where = s["pos"].double()[s["axis"]]
        turn = torch.polar(torch.ones((), dtype=torch.float64, device=DEV),
                           sign * where.transpose(0, 1) * freq).unsqueeze(1)
        out = []
        for x in (q, k):  # each pair as one complex number
            z = torch.complex(x[..., :D // 2].contiguous(), x[..., D // 2:].contiguous()) * turn
            out.append(torch.cat([z.real, z.imag], dim=-1))
        return tuple(out)
    full = 4.0 * D * q.shape[1] * sum(float(n) ** 2 for n in s["lens"])
    if full * (2.5 if case["op"] == "attn_bwd" else 1.0) > EXACT_FLOPS:
        return None
    forward = case["op"] == "attn_fwd"
    if forward:
        o, lse = torch.empty_like(q), torch.empty(q.shape[1], q.shape[0], dtype=torch.float64,
                                                  device=DEV)
    else:
        od, lsed, g = s["o"].double(), s["lse"].double(), s["do"].double()
        dq, dk, dv = torch.empty_like(q), torch.zeros_like(k), torch.zeros_like(v)
    start = 0
    for n in s["lens"]:
        rows = slice(start, start + n)
        hidden = torch.ones(n, n, dtype=torch.bool, device=DEV).triu(1) if s["causal"] else None
        for h in range(q.shape[1]):
            qh, kh, vh = q[rows, h], k[rows, h // G], v[rows, h // G]
            z = torch.einsum("id,jd->ij", qh, kh) / math.sqrt(D)
            if hidden is not None:
                z[hidden] = -math.inf
            if forward:
                norm = torch.logsumexp(z, dim=1)
                lse[h, rows] = norm
                o[rows, h] = torch.exp(z - norm[:, None]) @ vh
            else:
                p = torch.exp(z - lsed[h, rows][:, None])
                gh = g[rows, h]
                dv[rows, h // G] += torch.einsum("ij,id->jd", p, gh)
                mean = torch.einsum("id,id->i", gh, od[rows, h])
                ds = p * (torch.einsum("id,jd->ij", gh, vh) - mean[:, None]) / math.sqrt(D)
                dq[rows, h] = ds @ kh
                dk[rows, h // G] += torch.einsum("ij,id->jd", ds, qh)
        start += n
    return (o, lse) if forward else (dq, dk, dv)
