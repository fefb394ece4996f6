"""Attention with odd groups of heads over many sequences and with large groups,
against the 64-bit form inside the oracle's bars."""
import numpy as np
import pytest
import torch

from fine_tuning_gb300 import build, ftk
from test_attn_gpu import check, inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    ftk.library()
    yield
    assert ftk.device_status(clear=True) == 0


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("B,Hq,Hkv", [(129, 7, 1), (129, 6, 2), (140, 3, 3), (128, 7, 1)])
def test_odd_groups_over_many_sequences(B, Hq, Hkv, D):
    """More sequences than the length order takes, so that tiles are found by their
    slots, pairs of (row tile, head) across two row tiles among them."""
    lens = np.random.default_rng(B + Hq).integers(100, 401, B)
    lens[::7] = np.random.default_rng(B).integers(0, 4, len(lens[::7]))
    check(*inputs(tuple(int(n) for n in lens), Hq, Hkv, D, torch.bfloat16, lead=5, tail=9), True)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("Hq,Hkv,D,lens", [(40, 1, 64, (700, 90)), (64, 1, 128, (300, 1, 200)),
                                           (64, 2, 16, (150, 0, 129))])
def test_large_groups(Hq, Hkv, D, lens, causal):
    check(*inputs(lens, Hq, Hkv, D, torch.bfloat16, fused=True), causal)


@pytest.mark.slow
def test_an_item_of_more_than_a_second():
    """One CTA passes over 6,144 query heads of 38,912 tokens for the first key
    tile: 1.9M tile steps, some 3e9 cycles, where a single wait may take 2e9.  Only
    the first and the last head have a gradient: the others add exact zeros, so
    every result is that of a call with these two heads."""
    T, H, D = 38912, 6144, 8
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    q2, k, v, do2 = (torch.randn((T, h, D), generator=g, device="cuda").bfloat16()
                     for h in (2, 1, 1, 2))
    cu = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    o2, lse2 = ftk.attn_fwd(q2, k, v, cu)
    dq2, dk2, dv2 = ftk.attn_bwd(do2, q2, k, v, o2, lse2, cu)
    q = q2[:, :1].repeat(1, H, 1)
    q[:, -1] = q2[:, 1]
    lse = lse2[:1].repeat(H, 1)
    lse[-1] = lse2[1]
    do, o = torch.zeros_like(q), torch.zeros_like(q)
    for x, x2 in ((do, do2), (o, o2)):
        x[:, 0], x[:, -1] = x2[:, 0], x2[:, 1]
    dq, dk, dv = (torch.full_like(x, float("nan")) for x in (q, k, v))
    ftk.attn_bwd(do, q, k, v, o, lse, cu, dq=dq, dk=dk, dv=dv)
    assert ftk.device_status() == 0
    assert torch.equal(dk, dk2) and torch.equal(dv, dv2)
    assert torch.equal(dq[:, 0], dq2[:, 0]) and torch.equal(dq[:, -1], dq2[:, 1])
    assert not bool(dq[:, 1:-1].any())
