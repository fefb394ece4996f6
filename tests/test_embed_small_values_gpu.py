"""Values below the smallest normal number in the table's gradient: kept where it is
overwritten, and not so where it is added to."""
import pytest
import torch

from oracle import residual as R

pytestmark = pytest.mark.gpu
U, TINY = 2.0 ** -24, 2.0 ** -126


@pytest.mark.parametrize("H", [64, 61])
def test_subnormals(H):
    from fine_tuning_gb300 import ftk
    V, T = 40, 30
    g = torch.Generator(device="cuda").manual_seed(0)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    ids = torch.randperm(V, generator=g, device="cuda")[:T].to(torch.int32)  # one token a row
    scale = 2.0 ** (-130 + 10 * torch.arange(H, device="cuda") / H)          # 2^-130 to 2^-120
    dx, base = rand(T, H) * scale, rand(V, H) * scale
    base[:, ::3] = rand(V, H)[:, ::3]
    dx[:, ::6] = rand(T, H)[:, ::6]
    got = ftk.embed_bwd(dx, ids, V)
    assert torch.equal(got[ids.long()], dx)  # subnormal sums as they are
    dW = base.clone()
    ftk.embed_bwd(dx, ids, V, dW=dW, accumulate=True)
    ref = R.embed_bwd(dx, ids, V, base=base)[0]
    # an addend, what it is added to and the sum may each count as zero below 2^-126
    assert ((dW.cpu().double() - ref).abs() <= U * ref.abs() + 3 * TINY).all()
    rest = torch.ones(V, dtype=torch.bool, device="cuda")
    rest[ids.long()] = False
    assert torch.equal(dW[rest], base[rest])  # rows that no token names as they were
