"""The embedding lookup and its table's gradient on the GPU, against 64 bits."""
import pytest
import torch

from oracle import residual as R

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def ftk():
    from fine_tuning_gb300 import ftk as f
    return f


def rand(*shape, dtype=torch.float32, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda").to(dtype)


def token_ids(kind, T, V, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    if kind == "same":
        t = torch.full((T,), V // 2, device="cuda")
    elif kind == "none":
        t = torch.full((T,), -100, device="cuda")
    elif kind == "distinct":
        t = torch.randperm(max(T, V), generator=g, device="cuda")[:T]  # ids past V among them
    elif kind == "skewed":  # a few ids fill most of the batch
        t = (torch.rand(T, generator=g, device="cuda") ** 8 * V).long()
    else:  # "mixed": some outside [0, V), on both sides
        t = torch.randint(-V // 4 - 1, V + V // 4 + 1, (T,), generator=g, device="cuda")
    return t.to(torch.int32)


def close(got, ref, bar):
    bad = ~((got.cpu().double() - ref).abs() <= bar)
    assert not bad.any(), (int(bad.sum()), got.shape)


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("T, H, V", [(1, 1, 1), (1, 8, 5), (7, 3, 9), (64, 64, 100), (333, 896, 50),
                                     (5, 1001, 300), (40, 5120, 17), (3, 70000, 4)])
@pytest.mark.parametrize("scale", [1.0, 29.93])
def test_lookup(dtype, T, H, V, scale):
    W, ids = rand(V, H, dtype=DT[dtype]), token_ids("mixed", T, V)
    close(ftk().embed_fwd(W, ids, scale), *R.embed_fwd(W, ids, scale))


def test_lookup_of_views_and_extreme_ids():
    wide = rand(50, 200, dtype=torch.bfloat16)
    ids = torch.tensor([0, 49, 50, -1, 2 ** 31 - 1, -2 ** 31, 7], dtype=torch.int32, device="cuda")
    for a in (0, 8, 1):
        out = torch.full((7, 160), 3.0, device="cuda", dtype=torch.bfloat16)
        W = wide[:, a:a + 96]
        ftk().embed_fwd(W, ids, 2.0, x=out[:, 32:128])
        close(out[:, 32:128], *R.embed_fwd(W, ids, 2.0))
        assert (out[:, :32] == 3).all() and (out[:, 128:] == 3).all()
    assert ftk().embed_fwd(wide, ids[:0]).shape == (0, 200)


def test_lookup_past_31_bits():
    W = torch.zeros(2 ** 19 + 8, 4104, device="cuda", dtype=torch.bfloat16)
    W[-3:] = rand(3, 4104, dtype=torch.bfloat16)
    V = W.shape[0]
    ids = torch.tensor([V - 1, 0, V - 3], dtype=torch.int32, device="cuda")
    assert torch.equal(ftk().embed_fwd(W, ids), W[ids.long()])


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("kind", ["same", "none", "distinct", "skewed", "mixed"])
@pytest.mark.parametrize("T, H, V", [(1, 1, 1), (2, 8, 3), (15, 24, 600), (16, 7, 2), (17, 64, 1000),
                                     (300, 896, 40), (1025, 33, 70000), (5000, 72, 300)])
def test_gradient(dtype, kind, T, H, V):
    dx, ids = rand(T, H, dtype=DT[dtype]), token_ids(kind, T, V)
    got = ftk().embed_bwd(dx, ids, V, 1.5)
    close(got, *R.embed_bwd(dx, ids, V, 1.5))
    assert torch.equal(got, ftk().embed_bwd(dx, ids, V, 1.5))
    base = rand(V, H, seed=3)
    dW = base.clone()
    assert ftk().embed_bwd(dx, ids, V, 1.5, dW=dW, accumulate=True) is dW
    close(dW, *R.embed_bwd(dx, ids, V, 1.5, base))
    unseen = torch.ones(V, dtype=torch.bool, device="cuda")
    ok = ids[(ids >= 0) & (ids < V)].long()
    unseen[ok] = False
    assert torch.equal(dW[unseen], base[unseen])
    assert (got[unseen] == 0).all()


@pytest.mark.parametrize("T, H, V, kind", [(60000, 16, 151936, "skewed"), (40000, 8, 70000, "mixed"),
                                           (140001, 8, 511, "skewed"), (140001, 8, 512, "mixed"),
                                           (300000, 4, 2 ** 20, "mixed"), (9000, 8, 10, "same")])
def test_gradient_of_long_batches(T, H, V, kind):
    dx, ids = rand(T, H), token_ids(kind, T, V)
    close(ftk().embed_bwd(dx, ids, V), *R.embed_bwd(dx, ids, V))


def test_gradient_of_a_vocabulary_of_31_bits():
    V = 2 ** 31 - 1
    ids = torch.tensor([0, V - 1, 7, -1, V - 1, 2 ** 30], dtype=torch.int32, device="cuda")
    dx = rand(6, 1)
    dW = torch.full((V, 1), float("nan"), device="cuda")
    ftk().embed_bwd(dx, ids, V, dW=dW)
    assert torch.equal(dW[[0, 7, 2 ** 30], 0], dx[[0, 2, 5], 0])
    assert dW[V - 1, 0] == dx[1, 0] + dx[4, 0]
    assert int(torch.count_nonzero(dW)) == 4  # zeros, no NaN, in every other row
    ftk().embed_bwd(dx, ids, V, dW=dW, accumulate=True)
    assert dW[7, 0] == 2 * dx[2, 0] and int(torch.count_nonzero(dW)) == 4


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("T, H, V, kind", [(300, 1024, 151936, "skewed"), (4097, 1000, 151913, "mixed"),
                                           (333, 1001, 150001, "mixed"), (5, 1024, 151936, "none"),
                                           (70000, 1024, 200003, "distinct")])
def test_gradient_of_a_large_table(dtype, T, H, V, kind):
    # more zeros than are written beside the sort
    dx, ids = rand(T, H, dtype=DT[dtype]), token_ids(kind, T, V)
    dW = torch.full((V, H), float("nan"), device="cuda")
    ftk().embed_bwd(dx, ids, V, dW=dW)
    ok = ids[(ids >= 0) & (ids < V)].long()
    seen, place = torch.unique(ok, return_inverse=True)
    small = torch.full_like(ids, -1)
    small[(ids >= 0) & (ids < V)] = place.to(torch.int32)
    close(dW[seen], *R.embed_bwd(dx, small, max(1, seen.numel())) if seen.numel() else (dW[seen].cpu(), 0))
    dW[seen] = 0
    assert not dW.any()


@pytest.mark.parametrize("accumulate", [False, True])
def test_gradient_into_views(accumulate):
    ids = token_ids("mixed", 100, 30)
    for a, H in ((0, 64), (4, 64), (1, 64), (8, 61)):
        dx = rand(100, 200, dtype=torch.bfloat16)[:, a:a + H]
        buf = rand(30, 300, seed=1)
        was = buf.clone()
        ftk().embed_bwd(dx, ids, 30, dW=buf[:, a:a + H], accumulate=accumulate)
        close(buf[:, a:a + H], *R.embed_bwd(dx, ids, 30, base=was[:, a:a + H] if accumulate else None))
        assert torch.equal(buf[:, :a], was[:, :a]) and torch.equal(buf[:, a + H:], was[:, a + H:])


def test_refusals():
    from fine_tuning_gb300.ftk import FtkError
    dx, ids, W = rand(10, 16), token_ids("mixed", 10, 20), rand(20, 16)
    for call in (lambda: ftk().embed_fwd(W, ids, x=W[:10]), lambda: ftk().embed_fwd(W, ids, float("inf")),
                 lambda: ftk().embed_bwd(dx, ids, 20, float("nan")), lambda: ftk().embed_bwd(dx, ids, 0),
                 lambda: ftk().embed_bwd(W[:10], ids, 20, dW=W),
                 lambda: ftk().embed_bwd(dx, ids, 20, workspace=torch.empty(64, dtype=torch.uint8,
                                                                            device="cuda"))):
        with pytest.raises(FtkError):
            call()
    for call in (lambda: ftk().embed_bwd(dx, ids, 20, accumulate=True),
                 lambda: ftk().embed_bwd(dx[:9], ids, 20), lambda: ftk().embed_bwd(dx, ids.long(), 20),
                 lambda: ftk().embed_bwd(dx, ids, 20, dW=rand(20, 16, dtype=torch.bfloat16)),
                 lambda: ftk().embed_bwd(dx, ids, 20, dW=rand(16, 20).T),
                 lambda: ftk().embed_fwd(W, ids, x=rand(10, 8)), lambda: ftk().embed_fwd(W, ids.cpu())):
        with pytest.raises(ValueError):
            call()


def test_empty_batch():
    dx, ids = rand(0, 16), torch.empty(0, dtype=torch.int32, device="cuda")
    assert (ftk().embed_bwd(dx, ids, 9) == 0).all()
    base = rand(9, 16)
    assert torch.equal(ftk().embed_bwd(dx, ids, 9, dW=base.clone(), accumulate=True), base)


def test_sums_follow_the_tokens_order():
    # 2^24 + 1 + 1 + ... in fp32: the ones are lost one by one after the large term, kept before it
    n = 12
    dx = torch.ones(n, 8, device="cuda")
    ids = torch.zeros(n, dtype=torch.int32, device="cuda")
    dx[0] = 2.0 ** 24
    assert (ftk().embed_bwd(dx, ids, 1) == 2.0 ** 24).all()
    assert (ftk().embed_bwd(dx.flip(0), ids, 1) == 2.0 ** 24 + 12).all()  # 11 + 2^24, ties to even


def test_graphs_that_share_a_workspace():
    V, ws = 500, torch.empty(1 << 22, dtype=torch.uint8, device="cuda")
    cases = [(rand(n, 40, seed=n), token_ids("skewed", n, V, n)) for n in (700, 90)]
    graphs = []
    for dx, ids in cases:
        out = ftk().embed_bwd(dx, ids, V, workspace=ws)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            ftk().embed_bwd(dx, ids, V, dW=out, workspace=ws)
        graphs.append((g, out))
    for g, out in graphs + graphs[::-1]:
        out.fill_(float("nan"))
        g.replay()
    torch.cuda.synchronize()
    for (dx, ids), (_, out) in zip(cases, graphs):
        close(out, *R.embed_bwd(dx, ids, V))


def test_autograd_and_tied_head():
    from fine_tuning_gb300 import autograd
    W = rand(40, 64, dtype=torch.bfloat16).requires_grad_()
    ids = token_ids("mixed", 50, 40)
    g = rand(50, 64, dtype=torch.bfloat16, seed=2)
    x = autograd.embedding(W, ids, 8.0)
    x.backward(g)
    ref, bar = R.embed_bwd(g, ids, 40, 8.0)
    close(W.grad, ref, bar + 2.0 ** -8 * ref.abs())  # rounded to the weight's type
    # the head's gradient and the lookup's in one buffer
    h = ftk().embed_fwd(W.detach(), ids)
    y = token_ids("mixed", 50, 40, 5)
    loss, lse = ftk().cce_fwd(h, W.detach(), y)
    dh, dW = ftk().cce_bwd(h, W.detach(), y, lse, torch.ones(1, device="cuda"))
    head = dW.clone()
    ftk().embed_bwd(dh, ids, 40, dW=dW, accumulate=True)
    close(dW, *R.embed_bwd(dh, ids, 40, base=head))
