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
