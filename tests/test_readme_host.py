"""The readme's example of the residual stream, run as it is printed, with 64-bit
stand-ins for the library's calls, against torch's own gradient."""
import os
import re
from types import SimpleNamespace

import torch

from oracle import residual as R

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
T, H, V, P, SEED, STEP, EPS = 9, 16, 20, 0.1, 7, 3, 1e-6


def example() -> str:
    with open(os.path.join(ROOT, "README.md"), encoding="utf-8") as f:
        blocks = re.findall(r"```python\n(.*?)```", f.read(), re.S)
    (code,) = [b for b in blocks if "rmsnorm_block_bwd" in b]
    return code


def stand_in(seen):
    """ftk's calls in 64 bits; seen gets the offset of each dropout."""
    def embed_bwd(dx, ids, V, scale=1.0, dW=None, accumulate=False):
        g = R.embed_bwd(dx, ids, V, scale)[0]
        return dW.add_(g) if accumulate else dW.copy_(g)

    def drop(x, p, seed, offset=0, step=None):
        seen.append(offset)
        return R.dropout(x, p, seed, offset, int(step))[0]

    def block_fwd(x, res, w, eps, w_post=None, p=0.0, seed=0, offset=0, step=None):
        seen.append(offset)
        keep = R.keep_mask(*x.shape, p, seed, offset, int(step))
        (h, rp), _ = R.block_fwd(x, res, w, eps, w_post, keep=keep, p=p)
        (y, r), _ = R.block_y(h, w, eps)
        return h, y, r, rp

    def block_bwd(dy, dh, x, h, w, rstd, rstd_post=None, w_post=None, p=0.0, seed=0, offset=0,
                  step=None):
        seen.append(offset)
        keep = R.keep_mask(*x.shape, p, seed, offset, int(step))
        return R.block_bwd(dy, dh, x, h, w, rstd, rstd_post, w_post, keep=keep, p=p)[0]

    return SimpleNamespace(embed_fwd=lambda W, ids, scale=1.0: R.embed_fwd(W, ids, scale)[0],
                           embed_bwd=embed_bwd, dropout_fwd=drop, dropout_bwd=drop,
                           rmsnorm_block_fwd=block_fwd, rmsnorm_block_bwd=block_bwd)


def run():
    g = torch.Generator().manual_seed(0)
    rand = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    M, ids = 0.3 * rand(H, H), torch.randint(-3, V, (T,), generator=g, dtype=torch.int32)
    base = rand(V, H)
    seen = []
    names = {"ftk": stand_in(seen), "W": rand(V, H), "ids": ids, "H": H, "V": V, "seed": SEED,
             "step": torch.tensor([STEP]), "eps": EPS, "w": 1 + 0.1 * rand(H),
             "w_next": 1 + 0.1 * rand(H), "dn": rand(T, H), "dh": rand(T, H), "dW": base.clone(),
             "block": lambda s: s @ M, "block_bwd": lambda db: db @ M.T}
    given = dict(names)
    exec(example(), names)
    return names, given, base, seen


def test_the_examples_gradients():
    names, given, base, seen = run()
    fwd = seen[:2]  # the offsets of the lookup's dropout and of the joint's
    leaf = {n: given[n].clone().requires_grad_() for n in ("W", "w", "w_next")}
    there = given["ids"] >= 0
    s = torch.where(there[:, None], leaf["W"][given["ids"].clamp(0).long()] * H ** 0.5, 0.0)

    def drop(x, offset):
        return torch.where(R.keep_mask(T, H, P, SEED, offset, STEP), x * R.drop_scale(P), 0.0)

    def norm(x, w):
        return x * (x.square().mean(1, keepdim=True) + EPS) ** -0.5 * w

    s = drop(s, fwd[0])
    h = s + drop(norm(given["block"](s), leaf["w"]), fwd[1])
    n = norm(h, leaf["w_next"])
    loss = (h * given["dh"]).sum() + (n * given["dn"]).sum()
    ref = dict(zip(leaf, torch.autograd.grad(loss, list(leaf.values()))))
    for name, got in (("W", names["dW"] - base), ("w", names["dw"]), ("w_next", names["dw_next"])):
        assert (got - ref[name]).abs().max() <= 1e-10 * ref[name].abs().max(), name


def test_the_examples_masks_differ_between_dropouts_and_steps():
    seen = run()[3]
    a, b = seen[:2]
    assert sorted(seen) == sorted([a, a, b, b])  # each backward has its forward's
    assert abs(a - b) >= 2 ** 32  # more than the steps of any run
    masks = [R.keep_mask(64, 64, P, SEED, offset, step) for offset in (a, b) for step in (0, 1, 2)]
    for i, one in enumerate(masks):
        for other in masks[i + 1:]:
            # two independent masks agree in (1 - p)^2 + p^2 = 0.82 of the places; 64 x 64 places
            # have a standard deviation of 0.006
            assert (one == other).double().mean() < 0.9
