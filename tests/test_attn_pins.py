"""The attention oracle: values that can be checked by hand, its gradients
against differences of its own forward, and the rotation against a one-axis
rotation (no GPU)."""
import math

import pytest
import torch

from oracle import attention as A


def rnd(*shape, seed=0):
    g = torch.Generator()
    g.manual_seed(seed)
    return torch.randn(shape, generator=g, dtype=torch.float64)


def test_one_token_returns_its_value():
    q, k, v = rnd(1, 2, 4), rnd(1, 1, 4, seed=1), rnd(1, 1, 4, seed=2)
    o, lse, _, _ = A.attn_fwd(q, k, v, [0, 1], 0.5, True, "f32")
    assert torch.allclose(o[0, 1], v[0, 0], atol=1e-15)
    assert math.isclose(lse[1, 0].item(), 0.5 * float(q[0, 1] @ k[0, 0]), rel_tol=1e-14)


def test_equal_scores_average_the_keys_that_a_token_sees():
    q, k, v = torch.zeros(4, 1, 3), torch.zeros(4, 1, 3), rnd(4, 1, 3)
    o, lse, _, _ = A.attn_fwd(q, k, v, [0, 3, 4], 1.0, True, "f32")
    for i in range(3):
        assert torch.allclose(o[i, 0], v[:i + 1, 0].mean(0), atol=1e-15)
        assert math.isclose(lse[0, i].item(), math.log(i + 1), abs_tol=1e-15)
    assert torch.allclose(o[3, 0], v[3, 0])
    o, _, _, _ = A.attn_fwd(q, k, v, [0, 3, 4], 1.0, False, "f32")
    assert torch.allclose(o[:3, 0], v[:3, 0].mean(0).expand(3, 3), atol=1e-15)


def test_rows_of_no_sequence_are_marked():
    x = rnd(6, 1, 2)
    o, lse, _, _ = A.attn_fwd(x, x, x, [1, 1, 4], 1.0, True, "f32")
    assert torch.isnan(o[[0, 4, 5]]).all() and torch.isnan(lse[0, [0, 4, 5]]).all()
    assert not torch.isnan(o[1:4]).any()


@pytest.mark.parametrize("causal", [True, False])
def test_gradients_against_differences(causal):
    cu, scale = [0, 3, 8], 0.7
    q, k, v, do = rnd(8, 4, 3), rnd(8, 2, 3, seed=1), rnd(8, 2, 3, seed=2), rnd(8, 4, 3, seed=3)
    o, lse, _, _ = A.attn_fwd(q, k, v, cu, scale, causal, "f32")
    grads, bars = A.attn_bwd(do, q, k, v, o, lse, cu, scale, causal, "f32")
    for x, g in zip((q, k, v), grads):
        d, step = rnd(*x.shape, seed=9), 1e-6

        def f(e):
            args = [y + e * d if y is x else y for y in (q, k, v)]
            return float((A.attn_fwd(*args, cu, scale, causal, "f32")[0] * do).sum())

        assert math.isclose((f(step) - f(-step)) / (2 * step), float((g * d).sum()), rel_tol=1e-7,
                            abs_tol=1e-8)
    assert all(bool((b > 0).all()) for b in bars[1:])


def test_the_rotation_by_equal_axes_is_the_plain_one_and_its_backward_the_transpose():
    import numpy as np
    import oracle
    T, H, D, theta = 11, 2, 8, 1e4
    x = rnd(T, H, D).float()
    pos = torch.arange(T, dtype=torch.int32).repeat(3, 1)
    f = [theta ** (-2 * i / D) for i in range(D // 2)]
    y, _ = A.qk_mrope(x, pos, [0, 1, 2, 1], f, 1.0, "f32")
    ref, _ = oracle.qk_rope(x, x.clone(), np.asarray([0, T], np.int32), theta, +1)
    assert np.abs(y.numpy() - np.asarray(ref).reshape(T, H, D)).max() < 1e-12
    pos = torch.randint(-50, 50, (3, T), dtype=torch.int32)
    g = rnd(T, H, D, seed=4)
    y, _ = A.qk_mrope(x, pos, [0, 1, 2, 1], f, 1.0, "f32")
    z, _ = A.qk_mrope(g, pos, [0, 1, 2, 1], f, -1.0, "f32")
    assert math.isclose(float((y * g).sum()), float((x.double() * z).sum()), rel_tol=1e-12)
