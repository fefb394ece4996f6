"""Attention rows on their own: keys whose scores are all -inf, rows whose
neighbours hold large values, against the 64-bit form and bit for bit."""
import math

import pytest
import torch

from fine_tuning_gb300 import autograd, build, ftk
from oracle import attention as A

pytestmark = pytest.mark.gpu
DEV = "cuda"
CODE = {torch.float32: "f32", torch.bfloat16: "bf16"}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    ftk.library()
    yield
    assert ftk.device_status(clear=True) == 0


def rnd(shape, seed, dtype):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return torch.randn(shape, generator=g, device=DEV).to(dtype)


def seen_fwd(q, k, v, scale, seen, code):
    """(o, lse, their bars) of one sequence in 64 bits where row i attends to
    the keys of seen[i] alone: the bars of the oracle's forward, from the scores
    that are seen (one that is -inf has a weight of zero exactly)."""
    q, k, v = q.double(), k.double(), v.double()
    n, Hq, D = q.shape
    G, u, r = Hq // k.shape[1], A.U, A.R[code]
    o, ob = torch.empty_like(q), torch.empty_like(q)
    lse = torch.empty((Hq, n), dtype=torch.float64, device=q.device)
    lb = lse.clone()
    for h in range(Hq):
        qs, ks, vs = q[:, h], k[:, h // G], v[:, h // G]
        ks = torch.where(torch.isfinite(ks), ks, 0.0)  # components of keys that are not seen
        z = (scale * (qs @ ks.T)).masked_fill(~seen, -math.inf)
        mag = (scale * (qs.abs() @ ks.abs().T)).masked_fill(~seen, 0.0)
        norm = torch.logsumexp(z, 1)
        p = torch.exp(z - norm[:, None])
        far = (norm[:, None] - z).masked_fill(p == 0, 0.0).amax(1)
        es = (D + 3) * 2 * u * mag.amax(1) + u * z.amax(1).abs()
        e = 2 * es + (8 + 3 * far) * u + (n + 3) * 2 * u
        o[:, h] = p @ vs
        ob[:, h] = (r + 2 * e[:, None] + (n + 3) * 2 * u) * (p @ vs.abs()) + r * o[:, h].abs()
        lse[h] = norm
        lb[h] = e + 4 * u * (norm.abs() + math.log(n + 1))
    return o, lse, ob, lb


def within(name, got, ref, bar):
    off = (got.double() - ref).abs()
    assert bool(torch.isfinite(got).all()), name
    assert bool((off <= bar).all()), f"{name}: {float((off / bar).max()):.2f} of its bar"


@pytest.mark.parametrize("dtype,D", [(torch.bfloat16, 16), (torch.bfloat16, 64),
                                     (torch.bfloat16, 80), (torch.bfloat16, 128)])
def test_rows_with_overflowing_scores_beside_rows_without(dtype, D):
    """Even rows score -2.4e39 / sqrt(D), -inf in 32 bits, with the first 128 keys
    and see the rest; odd rows see all, and the second half of the first key tile
    scores far above their first half."""
    n, Hq, Hkv = 300, 4, 2
    q, k, v = (rnd((n, h, D), i, dtype) for i, h in enumerate((Hq, Hkv, Hkv)))
    q[0::2, :, 0], q[1::2, :, 0] = 8.0, 0.0
    k[:128, :, 0], k[128:, :, 0] = -3e38, 0.0
    q[:, :, 1] = 8.0
    k[:64, :, 1], k[64:128, :, 1], k[128:, :, 1] = 0.0, 20.0, -1.0
    scale = D ** -0.5
    seen = torch.ones(n, n, dtype=torch.bool, device=DEV)
    seen[0::2, :128] = False
    cu = torch.tensor([0, n], dtype=torch.int32, device=DEV)
    o, lse = ftk.attn_fwd(q, k, v, cu, causal=False)
    ro, rl, bo, bl = seen_fwd(q, k, v, scale, seen, CODE[dtype])
    within("o", o, ro, bo)
    within("lse", lse, rl, bl)
    # dk and dv (dq holds sums of the 3e38)
    do = rnd(q.shape, 9, dtype)
    grads = ftk.attn_bwd(do, q, k, v, o, lse, cu, causal=False)
    ref, bar = A.attn_bwd(do, q, k, v, o, lse, cu, scale, False, CODE[dtype])
    for name, g, r, b in list(zip(("dq", "dk", "dv"), grads, ref, bar))[1:]:
        within(name, g, r, b)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("dtype,D,first", [
    (torch.float32, 16, 40), (torch.float32, 64, 70), (torch.float32, 128, 130),
    (torch.float32, 256, 33), (torch.bfloat16, 33, 70), (torch.bfloat16, 160, 33),
    (torch.bfloat16, 64, 130), (torch.bfloat16, 128, 130), (torch.bfloat16, 128, 70)])
@pytest.mark.parametrize("n", [330, 1500])
def test_first_keys_with_infinite_components(dtype, D, first, causal, n):
    """Every key of the first tile scores -inf with every query, later ones are
    finite: they alone count.  (1,500 tokens take the 64-row tiles of the
    CUDA-core form, 330 its 32-row ones.)  With the causal mask the rows of the
    first keys themselves have nothing but -inf, and no value by the definition."""
    Hq, Hkv = 8, 4
    q, k, v = (rnd((n, h, D), i, dtype) for i, h in enumerate((Hq, Hkv, Hkv)))
    q[:, :, 0] = q[:, :, 0].abs() + 0.25
    k[:first, :, 0] = -math.inf
    seen = torch.ones(n, n, dtype=torch.bool, device=DEV)
    if causal:
        seen = seen.tril()
    seen[:, :first] = False
    cu = torch.tensor([0, n], dtype=torch.int32, device=DEV)
    o, lse = ftk.attn_fwd(q, k, v, cu, causal=causal)
    ro, rl, bo, bl = seen_fwd(q, k, v, D ** -0.5, seen, CODE[dtype])
    rows = slice(first if causal else 0, n)
    within("o", o[rows], ro[rows], bo[rows])
    within("lse", lse[:, rows], rl[:, rows], bl[:, rows])
    if causal:
        assert bool(torch.isnan(o[:first]).all()) and bool((lse[:, :first] == -math.inf).all())


def everything(q, k, v, do, cu, causal):
    o, lse = ftk.attn_fwd(q, k, v, cu, causal=causal)
    return [o, lse.T, *ftk.attn_bwd(do, q, k, v, o, lse, cu, causal=causal)]


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("dtype,D", [(torch.bfloat16, 64), (torch.bfloat16, 128),
                                     (torch.bfloat16, 24), (torch.bfloat16, 80),
                                     (torch.float32, 64)])
@pytest.mark.parametrize("n", [20, 100, 200, 330])
def test_large_values_of_other_sequences_change_no_bit(dtype, D, causal, n):
    """Rows behind a sequence's end hold large finite queries, keys and values, as
    another sequence or as padding; its own rows stay as they are."""
    T, Hq, Hkv = n + 230, 4, 2
    x = [rnd((T, h, D), i, dtype) for i, h in enumerate((Hq, Hkv, Hkv, Hq))]
    cu = torch.tensor([0, n], dtype=torch.int32, device=DEV)
    clean = [t[:n] for t in everything(*x, cu, causal)]
    for t in x:
        t[n:] *= 50
    both = torch.tensor([0, n, T], dtype=torch.int32, device=DEV)
    for c in (cu, both):
        for name, a, b in zip(("o", "lse", "dq", "dk", "dv"), clean, everything(*x, c, causal)):
            assert torch.equal(a, b[:n]), name


@pytest.mark.parametrize("dtype,D", [(torch.bfloat16, 64), (torch.bfloat16, 128),
                                     (torch.float32, 64)])
@pytest.mark.parametrize("cut", [10, 150, 205])
def test_later_tokens_of_a_causal_sequence_change_no_bit(dtype, D, cut):
    n, Hq, Hkv = 330, 4, 2
    x = [rnd((n, h, D), i, dtype) for i, h in enumerate((Hq, Hkv, Hkv, Hq))]
    cu = torch.tensor([0, n], dtype=torch.int32, device=DEV)
    clean = [t[:cut].clone() for t in everything(*x, cu, True)[:3]]
    for t in x[:3]:
        t[cut:] *= 50
    for name, a, b in zip(("o", "lse", "dq"), clean, everything(*x, cu, True)):
        assert torch.equal(a, b[:cut]), name


@pytest.mark.parametrize("D", [64, 128])
def test_a_row_does_not_depend_on_its_neighbours_queries(D):
    """Full mask: every second query grows until it raises its maximum in every
    tile; the others, and their gradients of q, stay as they are."""
    n = 400
    q, k, v, do = (rnd((n, 2, D), i, torch.bfloat16) for i in range(4))
    cu = torch.tensor([0, n], dtype=torch.int32, device=DEV)
    clean = [t[::2].clone() for t in everything(q, k, v, do, cu, False)[:3]]
    q[1::2] *= 60
    for name, a, b in zip(("o", "lse", "dq"), clean, everything(q, k, v, do, cu, False)):
        assert torch.equal(a, b[::2]), name


def test_a_workspace_with_gaps_is_refused():
    """Its elements' count says nothing about the bytes from its first one on."""
    q, k, v, do = (rnd((50, 2, 64), i, torch.bfloat16) for i in range(4))
    cu = torch.tensor([0, 50], dtype=torch.int32, device=DEV)
    o, lse = ftk.attn_fwd(q, k, v, cu)
    n = ftk.attn_bwd_workspace_bytes(50, 2, 2, 64, q.dtype)
    both = torch.zeros(n, 2, dtype=torch.uint8, device=DEV)
    with pytest.raises(ValueError):
        ftk.attn_bwd(do, q, k, v, o, lse, cu, workspace=both[:, 0])
    ftk.attn_bwd(do, q, k, v, o, lse, cu, workspace=both)
    with pytest.raises(ftk.FtkError):
        ftk.attn_bwd(do, q, k, v, o, lse, cu, workspace=both.view(-1)[:n - 1])


def test_two_threads_at_once_from_their_first_call_on():
    """The binding leaves the interpreter's lock during a call: each thread on its own
    stream gets the bits of a lone call."""
    import threading
    cases = []
    for i, D in enumerate((64, 128, 24, 96)):
        x = [rnd((700, h, D), i, torch.bfloat16) for h in (4, 2, 2, 4)]
        cases.append((x, torch.tensor([0, 300, 700], dtype=torch.int32, device=DEV)))
    torch.cuda.synchronize()
    got = [None] * len(cases)

    def work(i):
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(5):
                got[i] = everything(*cases[i][0], cases[i][1], True)
            torch.cuda.current_stream().synchronize()

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(cases))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    for (x, cu), g in zip(cases, got):
        for a, b in zip(g, everything(*x, cu, True)):
            assert torch.equal(a, b)


FORMS = [(torch.float32, 16), (torch.bfloat16, 64), (torch.bfloat16, 128), (torch.bfloat16, 33)]


@pytest.mark.parametrize("dtype,D", FORMS)
@pytest.mark.parametrize("bounds", [[3, 3], [0, 0, 0], [40, 40], [5] * 200])
def test_batches_whose_sequences_are_all_empty(dtype, D, bounds):
    q, k, v, do = (rnd((40, h, D), i, dtype) for i, h in enumerate((4, 2, 2, 4)))
    cu = torch.tensor(bounds, dtype=torch.int32, device=DEV)
    o, lse = torch.full_like(q, 7.0), torch.full((4, 40), 7.0, device=DEV)
    outs = [torch.full_like(t, 7.0) for t in (q, k, v)]
    ftk.attn_fwd(q, k, v, cu, o=o, lse=lse)
    ftk.attn_bwd(do, q, k, v, o, lse, cu, dq=outs[0], dk=outs[1], dv=outs[2])
    for t in (o, lse, *outs):
        assert bool((t == 7).all())
    leaves = [t.clone().requires_grad_(True) for t in (q, k, v)]
    out = autograd.attention(*leaves, cu)
    out.backward(do)
    assert not bool(out.any()) and not any(bool(t.grad.any()) for t in leaves)


@pytest.mark.parametrize("dtype,D", FORMS)
def test_one_tensor_as_queries_keys_and_values(dtype, D):
    x, do = rnd((150, 2, D), 0, dtype), rnd((150, 2, D), 1, dtype)
    cu = torch.tensor([0, 20, 150], dtype=torch.int32, device=DEV)
    apart = everything(x, x.clone(), x.clone(), do, cu, True)
    for a, b in zip(apart, everything(x, x, x, do, cu, True)):
        assert torch.equal(a, b)
    leaf = x.clone().requires_grad_(True)
    autograd.attention(leaf, leaf, leaf, cu).backward(do)
    ref = sum(t.double() for t in apart[2:])
    # two sums of rounded tensors: half a step of each operand and of each sum
    bar = 4 * A.R[CODE[dtype]] * sum(t.double().abs() for t in apart[2:])
    assert bool(((leaf.grad.double() - ref).abs() <= bar).all())


@pytest.mark.parametrize("D", [64, 128])
def test_one_sequence_among_many_empty_ones(D):
    """The items of 100,000 empty sequences are dropped on the device."""
    q, k, v, do = (rnd((300, h, D), i, torch.bfloat16) for i, h in enumerate((4, 2, 2, 4)))
    one = torch.tensor([0, 300], dtype=torch.int32, device=DEV)
    many = torch.cat([torch.zeros(50000, dtype=torch.int32), torch.full((50001,), 300)]).int().to(DEV)
    for name, a, b in zip(("o", "lse", "dq", "dk", "dv"), everything(q, k, v, do, one, True),
                          everything(q, k, v, do, many, True)):
        assert torch.equal(a, b), name


def test_two_graphs_that_share_a_workspace():
    """Replayed one after the other, each clobbers it and needs nothing of it."""
    sets, ref, graphs, outs = [], [], [], []
    ws = torch.empty(ftk.attn_bwd_workspace_bytes(300, 8, 2, 64, torch.bfloat16),
                     dtype=torch.uint8, device=DEV)
    for s in range(2):
        q, k, v, do = (rnd((300, h, 64), 10 * s + i, torch.bfloat16)
                       for i, h in enumerate((8, 2, 2, 8)))
        cu = torch.tensor([0, 50 + 100 * s, 300], dtype=torch.int32, device=DEV)
        o, lse = ftk.attn_fwd(q, k, v, cu)
        ref.append(ftk.attn_bwd(do, q, k, v, o, lse, cu))
        sets.append((do, q, k, v, o, lse, cu))
    torch.cuda.synchronize()
    for x in sets:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(ftk.attn_bwd(*x, workspace=ws))
        graphs.append(g)
    for _ in range(3):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    for a, b in zip(outs, ref):
        assert all(torch.equal(x, y) for x, y in zip(a, b))
