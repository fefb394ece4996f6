"""What the autograd wrappers hand to the backward pass (no GPU: the library's calls
are replaced by ones that note their arguments)."""
import numpy as np
import pytest
import torch

from fine_tuning_gb300 import autograd, ftk


def _mrope(q, k, tables):
    return autograd.qk_mrope(q, k, torch.zeros(3, 5, dtype=torch.int32), tables["axis_of"], 0.0,
                             tables["inv_freq"])


def _rope(q, k, tables):
    return autograd.qk_rope(q, k, torch.tensor([0, 5], dtype=torch.int32), 0.0, tables["inv_freq"])


def _norm_rope(q, k, tables):
    w = torch.ones(8)
    return autograd.qk_norm_rope(q, k, w, w, torch.tensor([0, 5], dtype=torch.int32), 1e-6, 0.0,
                                 tables["inv_freq"])


@pytest.mark.parametrize("kind", [np.array, list, torch.tensor])
@pytest.mark.parametrize("op", [_mrope, _rope, _norm_rope])
def test_host_tables_that_change_between_forward_and_backward(op, kind, monkeypatch):
    seen = []

    def note(*args, **kw):
        tables = [a for a in (*args, *kw.values())
                  if isinstance(a, (np.ndarray, list)) or
                  (isinstance(a, torch.Tensor) and a.dim() == 1 and a.numel() == 4)]
        seen.append([np.asarray(t).tolist() for t in tables])

    pair = lambda q, k, *a, **kw: (note(*a, **kw), (q, k))[1]  # noqa: E731
    for name in ("qk_mrope_fwd", "qk_mrope_bwd", "qk_rope_freq_fwd", "qk_rope_freq_bwd"):
        monkeypatch.setattr(ftk, name, pair)
    monkeypatch.setattr(ftk, "qk_norm_rope_fwd", lambda q, k, *a, **kw: (
        note(*a, **kw), (q.clone(), k.clone(), torch.ones(1), torch.ones(1)))[1])
    monkeypatch.setattr(ftk, "qk_norm_rope_bwd", lambda q, k, *a, **kw: (
        note(*a, **kw), (q, k, torch.ones(8), torch.ones(8)))[1])
    tables = {"axis_of": kind([0, 1, 2, 1]), "inv_freq": kind([1.0, 0.5, 0.25, 0.125])}
    q, k = torch.ones(5, 2, 8, requires_grad=True), torch.ones(5, 1, 8, requires_grad=True)
    q2, k2 = op(q * 1, k * 1, tables)
    for t in tables.values():
        t[0], t[1] = t[1] + 0, t[0] + 0
    (q2.sum() + k2.sum()).backward()
    assert len(seen) == 2 and seen[0] and seen[0] == seen[1]
