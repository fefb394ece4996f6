"""Measured cases of the residual stream around a decoder's blocks: the embedding
lookup that begins it and its gradient, dropout whose mask is never stored, and the
joint of a block's output with the stream (norm after the block, gate, dropout,
scales, residual add, norm before the next block) with its backward pass.

``run`` computes an operator in plain torch (``own`` false) or through the
library's calls (``own`` true), on the same state; ``exact`` restates the
definitions in 64 bits.  Shapes are those of ``fine_tuning_gb300.workloads``
or generic ones.

Definitions, for token row t and column j of [T, H] tensors:

    dropout    u[t, j]: the 16-bit number j & 7 (low half of a word first) of the
               128 bits that Philox4x32-10 (Salmon, Moraes, Dror and Shaw, SC 2011)
               makes of the key seed and the counter (j >> 3, t, offset + step)
               keep = u >= thr, thr = floor(65536 p + 1/2)
               y = keep ? x * 65536 / (65536 - thr) : 0     (backward: the same of dy)
    embedding  x[t] = scale * W[id[t]], 0 where id[t] lies outside [0, V)
               dW[v] = scale * sum over t with id[t] = v of dx[t]            (fp32)
    block      b = x r1 w_post gate[j] gate_tok[t],  r1 = 1 / sqrt(mean_j x^2 + eps)
               h = res_scale res + x_scale dropout(b)                    (stored)
               y = h r2 w,  r2 = 1 / sqrt(mean_j h^2 + eps)
               G = dh + r2 w dy - r2^3 h (sum_j dy w h) / H,  dres = res_scale G
               g = x_scale dropout(G),  e = g gate gate_tok
               dx = r1 w_post e - r1^3 x (sum_j e w_post x) / H
               dw = sum_t dy h r2,  S = sum_t g gate_tok x r1
               dw_post = gate S,  dgate = w_post S
               dgate_tok[t] = sum_j g gate w_post x r1
    (without w_post: r1 = w_post = 1 and no term in r1^3)
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-6
LOW = 0xFFFFFFFF


# ------------------------------------------------------------------ cases

def _drop(name, op, dtype, T, H, p, wide=False, step=False):
    case = {"op": op, "dtype": dtype, "T": T, "H": H, "p": p, "wide": wide, "step": step}
    return {"name": name, **case} if name else case


def _embed(name, op, dtype, T, H, V, scale, pad=0.0, parts=1):
    case = {"op": op, "dtype": dtype, "T": T, "H": H, "V": V, "scale": scale, "pad": pad,
            "parts": parts}
    return {"name": name, **case} if name else case


def _block(name, op, dtype, T, H, p=0.0, post=True, gate=False, tok=False, res_scale=1.0,
           x_scale=1.0, wide=False):
    case = {"op": op, "dtype": dtype, "T": T, "H": H, "p": p, "post": post, "gate": gate,
            "tok": tok, "res_scale": res_scale, "x_scale": x_scale, "wide": wide}
    return {"name": name, **case} if name else case


def listed():
    return [
        # the input of one adapter on four short sequences: what a call costs at least
        _drop("dropout-fwd-tiny-f32", "dropout_fwd", "f32", 64, 64, 0.05),
        # the adapters' input over a packed Qwen2.5-0.5B batch
        _drop("dropout-fwd-16384x896", "dropout_fwd", "bf16", 16384, 896, 0.1),
        # Qwen3-8B's stream, an odd number of tokens, the step counted on the device
        _drop("dropout-bwd-65535x4096", "dropout_bwd", "bf16", 65535, 4096, 0.1, step=True),
        # one short prompt through Llama-3.2-1B's table
        _embed("embed-fwd-333x2048", "embed_fwd", "bf16", 333, 2048, 128256, 1.0),
        # a packed Qwen3-8B batch with padding behind the last sequence
        _embed("embed-fwd-65536x4096", "embed_fwd", "bf16", 65536, 4096, 151936, 64.0, pad=0.02),
        # the table's whole gradient from one packed Qwen2.5-0.5B batch
        _embed("embed-bwd-16384x896", "embed_bwd", "bf16", 16384, 896, 151936, 1.0),
        # two micro-batches at Qwen3-32B's width, the second added to the first's gradient
        _embed("embed-bwd-2x32768x5120", "embed_bwd", "bf16", 65536, 5120, 151936, 1.0, pad=0.02,
               parts=2),
        # four short sequences in fp32, every term of the joint there
        _block("block-fwd-tiny-f32", "block_fwd", "f32", 64, 64, p=0.1, gate=True, tok=True,
               res_scale=0.7, x_scale=0.5),
        # Qwen3-8B's stream, norms on both sides of the block and dropout
        _block("block-fwd-65536x4096", "block_fwd", "bf16", 65536, 4096, p=0.1, x_scale=0.22),
        # rows whose length is odd, so that no row but the first is aligned
        _block("block-bwd-4095x1001", "block_bwd", "bf16", 4095, 1001, p=0.1, gate=True),
        # Qwen2.5-0.5B's stream: dropout and a learned gate for each channel, no norm behind
        _block("block-bwd-16384x896", "block_bwd", "bf16", 16384, 896, p=0.1, post=False,
               gate=True),
        # the largest: Qwen3-32B's width, every term of the joint there
        _block("block-bwd-65536x5120", "block_bwd", "bf16", 65536, 5120, p=0.1, gate=True,
               tok=True, x_scale=0.5),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["dropout_fwd", "dropout_bwd", "embed_fwd", "embed_bwd", "block_fwd",
                     "block_fwd", "block_bwd", "block_bwd"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    odd = rng.random() < 0.2
    H = rng.choice([64, 896, 2048, 4096, 5120, 8 * _log(rng, 1, 640)])
    if odd:
        H = _log(rng, 1, 2048)
    most = (1 << 25 if odd else 1 << 27) // H
    T = _log(rng, 1, max(2, min(most, 131072)))
    p = rng.choice([0.0, 0.05, 0.1, 0.1, 0.3, 0.5])
    if op.startswith("dropout"):
        return _drop("", op, dtype, T, H, p, wide=rng.random() < 0.3, step=rng.random() < 0.5)
    if op.startswith("embed"):
        return _embed("", op, dtype, T, H, _log(rng, 100, 151936), rng.choice([1.0, 0.5, 64.0]),
                      pad=rng.choice([0.0, 0.02, 0.3]),
                      parts=rng.choice([1, 1, 2]) if op == "embed_bwd" else 1)
    return _block("", op, dtype, T, H, p, post=rng.random() < 0.7, gate=rng.random() < 0.5,
                  tok=rng.random() < 0.4, res_scale=rng.choice([1.0, 1.0, 0.7]),
                  x_scale=rng.choice([1.0, 0.22]), wide=rng.random() < 0.2)


# ------------------------------------------------------------------ inputs

def _normal(gen, shape, dtype, std=1.0, mean=0.0):
    t = torch.empty(shape, dtype=torch.float32, device=DEV)
    t.normal_(mean, std, generator=gen)
    return t.to(dtype)


def _rows(gen, case, std=1.0):
    """[T, H] values; with wide, the left part of the rows of a wider projection."""
    T, H, dtype = case["T"], case["H"], TYPES[case["dtype"]]
    if case.get("wide"):
        return _normal(gen, (T, H + 64), dtype, std)[:, :H]
    return _normal(gen, (T, H), dtype, std)


def _frequencies(V):
    """How often the tokens of a vocabulary of V are met, by rank."""
    f = 1.0 / (np.arange(V) + 2.7)
    return f / f.sum()


def _token_ids(gen, case):
    T, V = case["T"], case["V"]
    ranks = torch.from_numpy(np.cumsum(_frequencies(V))).to(DEV)
    u = torch.rand(T, generator=gen, device=DEV, dtype=torch.float64)
    r = torch.searchsorted(ranks, u).clamp_(max=V - 1)
    ids = torch.randperm(V, generator=gen, device=DEV)[r].to(torch.int32)
    pad = int(T * case["pad"])
    if pad:
        ids[T - pad:] = -100
    return ids


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(int(seed) * 6151 + 29)
    op, T, H, dtype = case["op"], case["T"], case["H"], TYPES[case["dtype"]]
    s = {"case": dict(case)}
    if "p" in case:  # what the random numbers are made from
        s["seed"] = (int(seed) * 0x9E3779B97F4A7C15 + 12345) & 0xFFFFFFFFFFFFFFFF
        s["offset"] = 7
        s["step"] = torch.tensor([int(seed) + 3], dtype=torch.int64, device=DEV) \
            if case.get("step") else None
    if op.startswith("dropout"):
        s["x"] = _rows(gen, case)
        return s
    if op.startswith("embed"):
        s["ids"] = _token_ids(gen, case)
        if op == "embed_fwd":
            s["W"] = _normal(gen, (case["V"], H), dtype, 0.02)
        else:
            s["dx"] = _normal(gen, (T, H), dtype)
        return s
    s["x"], s["res"] = _rows(gen, case), _rows(gen, case, 2.0)
    s["w"] = _normal(gen, (H,), dtype, 0.1, 1.0)
    s["w_post"] = _normal(gen, (H,), dtype, 0.1, 1.0) if case["post"] else None
    s["gate"] = _normal(gen, (H,), dtype, 0.1, 0.5) if case["gate"] else None
    s["gate_tok"] = torch.sigmoid(_normal(gen, (T,), torch.float32)) if case["tok"] else None
    if op == "block_bwd":  # what the forward pass left, and the gradients that arrive
        out = _block_fwd(s)
        s["h"], s["rstd"] = out[0], out[2]
        s["rstd_post"] = out[3] if case["post"] else None
        s["dy"], s["dh"] = _normal(gen, (T, H), dtype), _normal(gen, (T, H), dtype)
        del s["res"]
    return s


# ------------------------------------------------------------------ plain forms

def _philox(key, c0, c1, c2, c3):
    """Four 32-bit words, in int64 tensors, of each counter."""
    k0, k1 = key & LOW, key >> 32
    for _ in range(10):
        a, b = c0 * 0xD2511F53, c2 * 0xCD9E8D57  # the low 64 bits; the shift's sign is masked off
        c0, c1, c2, c3 = ((b >> 32) & LOW) ^ c1 ^ k0, b & LOW, ((a >> 32) & LOW) ^ c3 ^ k1, a & LOW
        k0, k1 = (k0 + 0x9E3779B9) & LOW, (k1 + 0xBB67AE85) & LOW
    return c0, c1, c2, c3


def _threshold(p):
    return int(math.floor(65536.0 * p + 0.5))


def _keep(s):
    """The mask [T, H]."""
    T, H = s["case"]["T"], s["case"]["H"]
    j = torch.arange((H + 7) // 8, device=DEV)
    t = torch.arange(T, device=DEV)[:, None]
    at = torch.zeros(1, dtype=torch.int64, device=DEV) + s["offset"]
    if s["step"] is not None:
        at = at + s["step"]
    j, t = torch.broadcast_tensors(j, t)
    words = _philox(s["seed"], j, t, at & LOW, (at >> 32) & LOW)
    thr = _threshold(s["case"]["p"])
    keep = torch.empty((*j.shape, 8), dtype=torch.bool, device=DEV)
    for i, w in enumerate(words):
        keep[..., 2 * i] = (w & 0xFFFF) >= thr
        keep[..., 2 * i + 1] = (w >> 16) >= thr
    return keep.reshape(T, -1)[:, :H]


def _dropped(s, x):
    """Dropout of fp32 values [T, H]."""
    thr = _threshold(s["case"]["p"])
    if thr == 0:
        return x
    return torch.where(_keep(s), x * (65536.0 / (65536 - thr)), 0.0)


def _embed_bwd(s):
    V, H = s["case"]["V"], s["case"]["H"]
    ids = s["ids"].long()
    ids = torch.where((ids >= 0) & (ids < V), ids, V)
    dW = torch.zeros((V + 1, H), dtype=torch.float32, device=DEV)
    dW.index_add_(0, ids, s["dx"].float() * s["case"]["scale"])
    return dW[:V]


def _factor(s):
    """gate[j] * gate_tok[t], as far as they are there."""
    f = 1.0
    if s["gate"] is not None:
        f = f * s["gate"].float()
    if s["gate_tok"] is not None:
        f = f * s["gate_tok"][:, None]
    return f


def _block_fwd(s):
    c = s["case"]
    b = s["x"].float()
    r1 = None
    if s["w_post"] is not None:
        r1 = torch.rsqrt((b * b).mean(-1) + EPS)
        b = b * r1[:, None] * s["w_post"].float()
    b = _dropped(s, b * _factor(s))
    h = (c["res_scale"] * s["res"].float() + c["x_scale"] * b).to(s["x"].dtype)
    n = h.float()
    r2 = torch.rsqrt((n * n).mean(-1) + EPS)
    y = (n * r2[:, None] * s["w"].float()).to(h.dtype)
    return (h, y, r2) if r1 is None else (h, y, r2, r1)


def _block_bwd(s):
    c, dtype = s["case"], s["x"].dtype
    x, h, dy, w = s["x"].float(), s["h"].float(), s["dy"].float(), s["w"].float()
    H = x.shape[1]
    r2 = s["rstd"][:, None]
    dn = dy * w
    G = s["dh"].float() + r2 * dn - r2 ** 3 * h * ((dn * h).sum(-1, keepdim=True) / H)
    out = [None, (c["res_scale"] * G).to(dtype), (dy * h * r2).sum(0)]
    g = c["x_scale"] * _dropped(s, G)
    del G, dn
    e = g * _factor(s)
    gt = g if s["gate_tok"] is None else g * s["gate_tok"][:, None]
    if s["w_post"] is None:
        out[0] = e.to(dtype)
        S, n = (gt * x).sum(0), x
    else:
        r1, wp = s["rstd_post"][:, None], s["w_post"].float()
        ew = e * wp
        out[0] = (r1 * ew - r1 ** 3 * x * ((ew * x).sum(-1, keepdim=True) / H)).to(dtype)
        S, n = (gt * x * r1).sum(0), x * r1 * wp
        out.append(S if s["gate"] is None else S * s["gate"].float())
    if s["gate"] is not None:
        out.append(S if s["w_post"] is None else S * s["w_post"].float())
    if s["gate_tok"] is not None:
        out.append((g * n * (1.0 if s["gate"] is None else s["gate"].float())).sum(-1))
    return tuple(out)


def _own(s):
    from fine_tuning_gb300 import ftk
    c, op = s["case"], s["case"]["op"]
    if op.startswith("dropout"):
        drop = ftk.dropout_fwd if op == "dropout_fwd" else ftk.dropout_bwd
        return drop(s["x"], c["p"], s["seed"], offset=s["offset"], step=s["step"])
    if op == "embed_fwd":
        return ftk.embed_fwd(s["W"], s["ids"], scale=c["scale"])
    if op == "embed_bwd":
        dW, n = None, -(-c["T"] // c["parts"])
        for a in range(0, c["T"], n):
            dW = ftk.embed_bwd(s["dx"][a:a + n], s["ids"][a:a + n], c["V"], scale=c["scale"],
                               dW=dW, accumulate=a > 0)
        return dW
    terms = dict(w_post=s["w_post"], gate=s["gate"], gate_tok=s["gate_tok"],
                 res_scale=c["res_scale"], x_scale=c["x_scale"], p=c["p"], seed=s["seed"],
                 offset=s["offset"], step=s["step"])
    if op == "block_fwd":
        out = ftk.rmsnorm_block_fwd(s["x"], s["res"], s["w"], EPS, **terms)
    else:
        out = ftk.rmsnorm_block_bwd(s["dy"], s["dh"], s["x"], s["h"], s["w"], s["rstd"],
                                    s["rstd_post"], **terms)
    return tuple(o for o in out if o is not None)


def run(s):
    if own:
        return _own(s)
    op = s["case"]["op"]
    if op.startswith("dropout"):
        return _dropped(s, s["x"].float()).to(s["x"].dtype)
    if op == "embed_fwd":
        ids, W = s["ids"].long(), s["W"]
        there = (ids >= 0) & (ids < W.shape[0])
        rows = W[torch.where(there, ids, 0)].float() * s["case"]["scale"]
        return torch.where(there[:, None], rows, 0.0).to(W.dtype)
    if op == "embed_bwd":
        return _embed_bwd(s)
    return _block_fwd(s) if op == "block_fwd" else _block_bwd(s)


# ------------------------------------------------------------------ cost, definition

def _distinct(n, V):
    """Rows of the table that n tokens touch, on average."""
    return float(-np.expm1(n * np.log1p(-_frequencies(V))).sum())


def work(case):
    """Bytes: each input read and each output written once.  Operations: one a
    product or sum of the formulas, for each element."""
    op, T, H = case["op"], case["T"], case["H"]
    es = 2 if case["dtype"] == "bf16" else 4
    n = T * H
    if op.startswith("dropout"):
        return {"bytes": 2 * n * es, "flops": n}
    if op.startswith("embed"):
        V, live = case["V"], T - int(T * case["pad"])
        if op == "embed_fwd":
            return {"bytes": n * es + int(_distinct(live, V)) * H * es + 4 * T, "flops": n}
        part = -(-T // case["parts"])
        total = live * H * es + 4 * T + 4 * V * H
        if case["parts"] == 2:  # the rows that the second part adds to are read and written again
            total += 8 * H * int(_distinct(max(0, live - part), V))
        return {"bytes": total, "flops": 2 * live * H}
    rows = 4 * T * (1 + case["post"] + case["tok"])
    cols = H * es * (1 + case["post"] + case["gate"])
    if op == "block_fwd":
        return {"bytes": 4 * n * es + rows + cols, "flops": 11 * n}
    return {"bytes": 6 * n * es + rows + cols + 4 * T * case["tok"]
            + 4 * H * (1 + case["post"] + case["gate"]), "flops": 30 * n}


def _mask64(s):
    """The mask from products of 16-bit halves, a chunk of rows at a time."""
    T, H, thr = s["case"]["T"], s["case"]["H"], _threshold(s["case"]["p"])
    at = s["offset"] + (0 if s["step"] is None else int(s["step"]))

    def wide(m, v):  # the high and low words of the 64-bit product m v
        m1, m0, v1, v0 = m >> 16, m & 0xFFFF, v >> 16, v & 0xFFFF
        low = m0 * v0
        mid = m1 * v0 + (low >> 16)
        mid2 = m0 * v1 + (mid & 0xFFFF)
        return m1 * v1 + (mid >> 16) + (mid2 >> 16), ((mid2 & 0xFFFF) << 16) | (low & 0xFFFF)

    out = []
    for a in range(0, T, 8192):
        rows = min(8192, T - a)
        ctr = [torch.arange((H + 7) // 8, device=DEV).repeat(rows, 1),
               (torch.arange(rows, device=DEV) + a)[:, None].repeat(1, (H + 7) // 8)]
        ctr += [torch.full_like(ctr[0], at & LOW), torch.full_like(ctr[0], (at >> 32) & LOW)]
        for i in range(10):
            k0 = ((s["seed"] & LOW) + i * 0x9E3779B9) & LOW
            k1 = ((s["seed"] >> 32) + i * 0xBB67AE85) & LOW
            h0, l0 = wide(0xD2511F53, ctr[0])
            h1, l1 = wide(0xCD9E8D57, ctr[2])
            ctr = [h1 ^ ctr[1] ^ k0, l1, h0 ^ ctr[3] ^ k1, l0]
        halves = torch.stack([v for c in ctr for v in (c % 65536, c // 65536)], dim=-1)
        out.append((halves >= thr).reshape(rows, -1)[:, :H])
    return torch.cat(out)


def exact(case, seed):
    s = prepare(case, seed)
    op, T, H = case["op"], case["T"], case["H"]
    if "p" in case:
        thr = _threshold(case["p"])
        m = _mask64(s).double().mul_(65536.0 / (65536 - thr)) if thr else \
            torch.ones((), dtype=torch.float64, device=DEV)
    if op.startswith("dropout"):
        return s["x"].double().mul_(m)
    if op.startswith("embed"):
        V = case["V"]
        ids = s["ids"].long()
        if op == "embed_fwd":
            table = torch.cat([s["W"], torch.zeros_like(s["W"][:1])])
            ids[(ids < 0) | (ids >= V)] = V
            return table[ids].double().mul_(case["scale"])
        t = torch.nonzero((ids >= 0) & (ids < V))[:, 0]
        where = torch.sparse_coo_tensor(torch.stack([ids[t], t]),
                                        torch.full((t.numel(),), float(case["scale"]),
                                                   dtype=torch.float64, device=DEV), (V, T))
        dW = torch.empty((V, H), dtype=torch.float64, device=DEV)
        for a in range(0, H, 512):
            dW[:, a:a + 512] = torch.sparse.mm(where, s["dx"][:, a:a + 512].double())
        return dW

    def d(name):
        return None if s.get(name) is None else s[name].double()

    x, w, wp, gate, tok = d("x"), d("w"), d("w_post"), d("gate"), d("gate_tok")
    gate = torch.ones_like(w) if gate is None else gate
    tok = torch.ones(T, dtype=torch.float64, device=DEV) if tok is None else tok
    if op == "block_fwd":
        r1 = torch.ones_like(tok) if wp is None else (x.square().mean(1) + EPS) ** -0.5
        b = torch.einsum("tj,t,j->tj", x, r1 * tok, gate * (1.0 if wp is None else wp))
        h = b.mul_(m).mul_(case["x_scale"]).add_(d("res"), alpha=case["res_scale"])
        n = h.to(s["x"].dtype).double()  # the norm is of the stored values
        r2 = (n.square().mean(1) + EPS) ** -0.5
        y = torch.einsum("tj,t,j->tj", n, r2, w)
        return (h, y, r2) if wp is None else (h, y, r2, r1)
    h, dy, r2 = d("h"), d("dy"), d("rstd")
    dot = torch.einsum("tj,j,tj->t", dy, w, h)
    G = d("dh") + torch.einsum("tj,t,j->tj", dy, r2, w) - (r2 ** 3 * dot / H)[:, None] * h
    dw = torch.einsum("tj,tj,t->j", dy, h, r2)
    del dy, h
    g = G * m * case["x_scale"]
    dres = G.mul_(case["res_scale"])
    r1 = torch.ones_like(tok) if wp is None else d("rstd_post")
    wpost = torch.ones_like(w) if wp is None else wp
    per_col = torch.einsum("tj,tj,t->j", g, x, tok * r1)
    per_row = torch.einsum("tj,tj,j->t", g, x, gate * wpost)
    dx = torch.einsum("tj,t,j->tj", g, tok * r1, gate * wpost)
    if wp is not None:
        dx -= (r1 ** 3 * tok * per_row / H)[:, None] * x
    out = [dx, dres, dw]
    if wp is not None:
        out.append(per_col * gate)
    if case["gate"]:
        out.append(per_col * wpost)
    if case["tok"]:
        out.append(per_row * r1)
    return tuple(out)
