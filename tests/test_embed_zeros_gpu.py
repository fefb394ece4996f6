"""The zeros of the overwritten table's gradient: every way that the kernels share them out."""
import pytest
import torch

from test_embed_gpu import close, ftk, rand, token_ids
from oracle import residual as R

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T, H, V", [
    (20000, 8, 1), (20000, 8, 33), (9000, 24, 100), (3000, 64, 16383), (3000, 61, 16385),
    # beside the sums as well, and not any more one token later
    (4085, 3080, 20011), (4086, 3080, 20011)])
def test_small_and_large_tables(T, H, V):
    ids = token_ids("mixed", T, V)
    dx = rand(T, H, dtype=torch.bfloat16)
    dW = torch.full((V, H), float("nan"), device="cuda")
    ftk().embed_bwd(dx, ids, V, dW=dW)
    close(dW, *R.embed_bwd(dx, ids, V))


@pytest.mark.parametrize("T", [0, 12 << 20])
def test_more_rows_than_the_first_ctas_mark(T):
    # 2^26 words of 32 rows: 8,192 words for each of 8,192 CTAs, all beside the sort
    V = 2 ** 31 - 1
    g = torch.Generator(device="cuda").manual_seed(3)
    ids = torch.randint(0, V, (T,), generator=g, device="cuda", dtype=torch.int32)
    dW = torch.full((V, 1), float("nan"), device="cuda")
    ftk().embed_bwd(torch.ones(T, 1, device="cuda"), ids, V, dW=dW)
    seen, count = torch.unique(ids, return_counts=True)
    assert torch.equal(dW[seen.long(), 0], count.float())
    assert int(torch.count_nonzero(dW)) == seen.numel()  # NaN counts, zeros do not
