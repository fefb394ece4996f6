"""What the autograd wrapper of a block's joint gives back (no GPU: the library's calls
are replaced by ones that make results of the documented shapes)."""
import pytest
import torch

from fine_tuning_gb300 import autograd, ftk

T, H = 5, 8


@pytest.fixture
def calls(monkeypatch):
    def fwd(x, res, w, eps, w_post=None, gate=None, gate_tok=None, *numbers):
        return x + res, x * 1, torch.ones(T), None if w_post is None else torch.ones(T)

    def bwd(dy, dh, x, h, w, rstd, rstd_post=None, w_post=None, gate=None, gate_tok=None, *numbers):
        some = lambda t, n: None if t is None else torch.arange(n, dtype=torch.float32)  # noqa: E731
        return dy * 1, dh * 1, some(w, H), some(w_post, H), some(gate, H), some(gate_tok, T)

    monkeypatch.setattr(ftk, "rmsnorm_block_fwd", fwd)
    monkeypatch.setattr(ftk, "rmsnorm_block_bwd", bwd)


@pytest.mark.parametrize("flat", [True, False])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_gradients_have_their_factors_shapes(calls, flat, dtype):
    # the binding takes any contiguous factor of H (or T) values: [1, H], and a gate of [T, 1],
    # as a projection to one feature makes it
    row, col = ((H,), (T,)) if flat else ((1, H), (T, 1))
    leaf = lambda shape, dt=dtype: torch.ones(shape, dtype=dt, requires_grad=True)  # noqa: E731
    x, res, w, wp, gate = leaf((T, H)), leaf((T, H)), leaf(row), leaf(row), leaf(row)
    tok = leaf(col, torch.float32)
    h, y = autograd.rmsnorm_block(x, res, w, 1e-6, wp, gate, tok)
    (h.sum() + y.sum()).backward()
    for t, n in ((w, H), (wp, H), (gate, H), (tok, T)):
        assert t.grad.dtype == t.dtype and torch.equal(t.grad.flatten(), torch.arange(n).to(t.dtype))
    assert x.grad.shape == res.grad.shape == (T, H)
