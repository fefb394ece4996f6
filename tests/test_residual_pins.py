"""The 64-bit oracle of the residual stream's operators, pinned on the CPU: the
generator against its authors' published vectors, gradients against differences."""
import math

import numpy as np
import pytest
import torch

from oracle import residual as R


@pytest.mark.parametrize("counter, key, out", [
    ((0, 0, 0, 0), (0, 0), (0x6627e8d5, 0xe169c58d, 0xbc57ac4c, 0x9b00dbd8)),
    ((0xffffffff,) * 4, (0xffffffff,) * 2, (0x408f276d, 0x41c83b0e, 0xa20bc7c6, 0x6d5451fd)),
    ((0x243f6a88, 0x85a308d3, 0x13198a2e, 0x03707344), (0xa4093822, 0x299f31d0),
     (0xd16cfe09, 0x94fdcceb, 0x5001e420, 0x24126ea1)),
])
def test_generator_known_answers(counter, key, out):
    assert tuple(int(v) for v in R.philox4x32(counter, key)) == out


def test_mask_counts_and_independence():
    T, H = 512, 512
    for p in (0.0, 0.1, 0.5, 0.97, 1.0):
        keep = R.keep_mask(T, H, p, seed=11)
        q = 1 - R.threshold(p) / 65536
        assert abs(keep.double().mean().item() - q) <= 5 * math.sqrt(q * (1 - q) / (T * H))
    a, b = R.keep_mask(T, H, 0.5, seed=11), R.keep_mask(T, H, 0.5, seed=11, offset=1)
    assert abs((a == b).double().mean().item() - 0.5) < 0.01
    # offset and step are one number; rows and columns do not depend on the sizes
    assert torch.equal(R.keep_mask(T, H, 0.5, 11, 3, 4), R.keep_mask(T, H, 0.5, 11, 7))
    assert torch.equal(a[:100, :77], R.keep_mask(100, 77, 0.5, 11))


def test_thresholds():
    assert [R.threshold(p) for p in (0.0, 2.0 ** -18, 2.0 ** -17, 0.5, 1.0)] == [0, 0, 1, 32768, 65536]
    assert R.drop_scale(1.0) == 0.0 and R.drop_scale(0.5) == 2.0


@pytest.mark.parametrize("post, gate, tok", [(1, 1, 1), (1, 0, 0), (0, 1, 0), (0, 0, 1), (0, 0, 0)])
@pytest.mark.parametrize("p", [0.0, 0.4])
def test_block_gradient_against_differences(post, gate, tok, p):
    T, H, eps, a, c = 3, 10, 1e-3, 0.7, 0.4
    g = torch.Generator().manual_seed(5)
    rand = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)
    x, res, w = rand(T, H), rand(T, H), 1 + 0.1 * rand(H)
    f = {"w_post": 1 + 0.1 * rand(H) if post else None, "gate": rand(H) if gate else None,
         "gate_tok": rand(T) if tok else None}
    keep = R.keep_mask(T, H, p, 3) if p else None
    dy, dh = rand(T, H), rand(T, H)

    def out(x, res, w, w_post, gate, gate_tok):
        (h, r1), _ = R.block_fwd(x, res, w, eps, w_post, gate, gate_tok, a, c, keep, p)
        (y, r), _ = R.block_y(h, w, eps)
        return h, y, r1, r

    def loss(**kw):
        v = dict(x=x, res=res, w=w, **f)
        v.update(kw)
        h, y, _, _ = out(**v)
        return ((dh * h).sum() + (dy * y).sum()).item()

    h, _, r1, r = out(x, res, w, **f)
    (dx, dres, dw, dwp, dg, dt), _ = R.block_bwd(dy, dh, x, h, w, r, r1, f["w_post"], f["gate"],
                                                 f["gate_tok"], a, c, keep, p)
    for name, value, grad in (("x", x, dx), ("res", res, dres), ("w", w, dw),
                              ("w_post", f["w_post"], dwp), ("gate", f["gate"], dg),
                              ("gate_tok", f["gate_tok"], dt)):
        assert (value is None) == (grad is None)
        if value is None:
            continue
        for _ in range(3):  # along random directions, central differences of step 1e-5
            v = rand(*value.shape)
            num = (loss(**{name: value + 1e-5 * v}) - loss(**{name: value - 1e-5 * v})) / 2e-5
            # third derivatives times 1e-10, and 64-bit rounding over the step: both below 1e-7
            assert abs(num - (grad * v).sum().item()) <= 1e-6 * (1 + abs(num)), name


def test_embedding_gradient_is_the_transpose():
    g = torch.Generator().manual_seed(2)
    W, dx = torch.randn(9, 4, generator=g), torch.randn(30, 4, generator=g)
    ids = torch.randint(-2, 11, (30,), generator=g, dtype=torch.int32)
    x, _ = R.embed_fwd(W, ids, 0.5)
    dW, _ = R.embed_bwd(dx, ids, 9, 0.5)
    assert abs((x * dx.double()).sum() - (dW * W.double()).sum()) < 1e-12
    assert np.all(x[(ids < 0) | (ids >= 9)].numpy() == 0)
    base = torch.randn(9, 4, generator=g)
    assert torch.allclose(R.embed_bwd(dx, ids, 9, 0.5, base)[0], dW + base.double())
