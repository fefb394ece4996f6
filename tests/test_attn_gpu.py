"""Attention over packed sequences on the GPU against the 64-bit form, inside
the bars that oracle/attention.py derives, and the calls around it: strides,
boundaries, foreign infinities, guards, streams, captured graphs, autograd."""
import math

import numpy as np
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


def rnd(shape, seed, dtype, std=1.0):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return (std * torch.randn(shape, generator=g, device=DEV)).to(dtype)


def inputs(lens, Hq, Hkv, D, dtype, fused=False, seed=0, lead=0, tail=0):
    """q, k, v, cu; `lead` and `tail` rows belong to no sequence."""
    T = lead + sum(lens) + tail
    if fused:
        x = rnd((T, Hq + 2 * Hkv, D), seed, dtype)
        q, k, v = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
    else:
        q, k, v = (rnd((T, h, D), seed + i, dtype) for i, h in enumerate((Hq, Hkv, Hkv)))
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lens)]) + lead, dtype=torch.int32, device=DEV)
    return q, k, v, cu


def within(name, got, ref, bar):
    got = got.double()
    assert torch.equal(torch.isnan(got), torch.isnan(ref)), name
    off = ((got - ref).abs() - bar).nan_to_num(-1.0)
    worst = ((got - ref).abs() / bar).nan_to_num(0.0).max() if got.numel() else 0
    assert bool((off <= 0).all()), f"{name}: {float(worst):.2f} of its bar"


def check(q, k, v, cu, causal, scale=None, seed=50, backward=True):
    code, D = CODE[q.dtype], q.shape[2]
    s = D ** -0.5 if scale is None else scale
    nan = lambda x: torch.full(x.shape, math.nan, dtype=x.dtype, device=DEV)  # noqa: E731
    o, lse = ftk.attn_fwd(q, k, v, cu, scale=scale, causal=causal, o=nan(q),
                          lse=torch.full((q.shape[1], q.shape[0]), math.nan, device=DEV))
    ro, rl, bo, bl = A.attn_fwd(q, k, v, cu, s, causal, code)
    within("o", o, ro, bo)
    within("lse", lse, rl, bl)
    if not backward:
        return
    do = rnd(q.shape, seed, q.dtype)
    # rows of no sequence: what stands there is not read into any other row
    dq, dk, dv = ftk.attn_bwd(do, q, k, v, o, lse, cu, scale=scale, causal=causal, dq=nan(q),
                              dk=nan(k), dv=nan(v))
    ref, bar = A.attn_bwd(do, q, k, v, o, lse, cu, s, causal, code)
    for n, g, r, b in zip(("dq", "dk", "dv"), (dq, dk, dv), ref, bar):
        within(n, g, r, b)


LENS = [(1,), (5, 17, 32, 10), (128,), (129,), (127, 1, 0, 300), (0, 0, 64, 0), (513, 2, 256),
        (1,) * 40, (255, 383, 64)]


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("dtype,Hq,Hkv,D", [
    (torch.float32, 4, 2, 16), (torch.float32, 3, 1, 64), (torch.float32, 2, 2, 128),
    (torch.float32, 2, 1, 256), (torch.float32, 2, 2, 33), (torch.float32, 1, 1, 1),
    (torch.bfloat16, 4, 2, 33), (torch.bfloat16, 2, 1, 160), (torch.bfloat16, 2, 2, 6)])
def test_cuda_core_forms(dtype, Hq, Hkv, D, causal):
    for i, lens in enumerate(LENS):
        check(*inputs(lens, Hq, Hkv, D, dtype, fused=i % 2 == 0, seed=i), causal)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("dtype,Hq,Hkv,D", [(torch.float32, 6, 2, 64), (torch.float32, 6, 6, 20),
                                            (torch.float32, 8, 2, 128), (torch.bfloat16, 6, 3, 33)])
def test_cuda_core_forms_that_fill_the_gpu(dtype, Hq, Hkv, D, causal):
    """Enough tiles for the larger tile of these kernels."""
    check(*inputs((700, 1, 513, 64, 0, 400), Hq, Hkv, D, dtype, fused=True), causal)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("Hq,Hkv,D", [(14, 2, 64), (4, 1, 64), (2, 2, 128), (8, 2, 128), (5, 1, 128),
                                      (3, 3, 80), (2, 1, 8), (4, 2, 16), (1, 1, 120), (6, 2, 72),
                                      (7, 1, 96), (1, 1, 64)])
def test_bf16(Hq, Hkv, D, causal):
    for i, lens in enumerate(LENS):
        check(*inputs(lens, Hq, Hkv, D, torch.bfloat16, fused=i % 2 == 0, seed=i), causal)


@pytest.mark.parametrize("D", [64, 128])
def test_longer_sequences(D):
    check(*inputs((2000, 77, 1031), 4, 2, D, torch.bfloat16, fused=True), True)
    check(*inputs((1500, 640), 2, 1, D, torch.bfloat16), False)


@pytest.mark.parametrize("dtype,D", [(torch.float32, 32), (torch.bfloat16, 64), (torch.bfloat16, 128)])
def test_large_scores_move_the_running_maximum(dtype, D):
    """Scores that grow along the keys, so that every tile raises the maximum."""
    q, k, v, cu = inputs((700, 130), 2, 1, D, dtype)
    ramp = torch.linspace(0.2, 3.0, q.shape[0], device=DEV)[:, None, None]
    k = (k.float().abs() * ramp).to(dtype)
    q = q.float().abs().to(dtype)
    check(q, k, v, cu, True, scale=0.25)
    check(q, k.flip(0), v, cu, False, scale=0.25)


@pytest.mark.parametrize("dtype,D", [(torch.float32, 16), (torch.bfloat16, 64), (torch.bfloat16, 128),
                                     (torch.bfloat16, 80)])
def test_rows_of_no_sequence_and_foreign_infinities(dtype, D):
    """Rows before, behind and between do not change what a sequence gets,
    whatever they hold, and are left as they were."""
    lens = (100, 200, 30)
    q, k, v, cu = inputs(lens, 4, 2, D, dtype, lead=3, tail=70)
    do = rnd(q.shape, 9, dtype)
    T = q.shape[0]

    def run(cu, x, cut):
        o, lse = ftk.attn_fwd(*x[:3], cu, o=torch.full_like(x[0], 7.0),
                              lse=torch.full((4, T), 7.0, device=DEV))
        outs = [torch.full_like(t, 7.0) for t in x[:3]]
        ftk.attn_bwd(x[3], *x[:3], o, lse, cu, dq=outs[0], dk=outs[1], dv=outs[2])
        for t in (o, lse.T, *outs):
            assert bool((t[:3] == 7).all()) and bool((t[T - 70:] == 7).all())
            assert not bool((t[cut] == 7).all())
        return [t[cut].clone() for t in (o, lse.T, *outs)]

    first, last = slice(3, 103), slice(303, 333)
    clean = [run(cu, (q, k, v, do), c) for c in (first, last)]
    dirty = [t.clone() for t in (q, k, v, do)]
    for t, bad in zip(dirty, (math.nan, math.inf, -math.inf, math.nan)):
        t[:3] = bad
        t[103:303] = bad
        t[T - 70:] = bad
    again = [run(cu, dirty, c) for c in (first, last)]
    for x, y in zip(clean, again):
        for a, b in zip(x, y):
            assert torch.equal(a, b)


def test_strides_alignment_and_wide_rows():
    q, k, v, cu = inputs((65, 130), 2, 1, 64, torch.bfloat16)
    ref, lse = ftk.attn_fwd(q, k, v, cu)
    # one element off a 16-byte boundary and odd row strides: the CUDA-core form
    off = torch.empty(195 * 131 + 1, dtype=torch.bfloat16, device=DEV)[1:].view(195, 131)
    qo = off[:, :128].view(195, 2, 64) if False else off.as_strided((195, 2, 64), (131, 64, 1), 1)
    qo.copy_(q)
    check(qo, k, v, cu, True)
    # a stride of its own for every tensor, on the tensor cores
    wide = [torch.zeros(195, 512, dtype=torch.bfloat16, device=DEV) for _ in range(4)]
    views = [w.as_strided((195, h, 64), (512, 64, 1), 64 * i)
             for i, (w, h) in enumerate(zip(wide, (2, 1, 1, 2)))]
    for x, y in zip(views, (q, k, v)):
        x.copy_(y)
    o2, lse2 = ftk.attn_fwd(*views[:3], cu, o=views[3])
    assert torch.equal(o2, ref) and torch.equal(lse2, lse)
    assert int((wide[3] != 0).any(0).sum()) <= 128  # nothing beside o's columns
    with pytest.raises(ValueError):
        ftk.attn_fwd(q.transpose(0, 1).contiguous().transpose(0, 1), k, v, cu)


@pytest.mark.parametrize("D", [64, 24])
def test_offsets_past_32_bits(D):
    """Row strides so large that byte and element offsets pass 2^31 (and 2^32)."""
    rows, ld = 300, 1 << 24
    big = torch.empty(rows * ld, dtype=torch.bfloat16, device=DEV)  # 10 GB, mostly untouched
    H = 2
    views = [big.as_strided((rows, H, D), (ld, D, 1), i * H * D) for i in range(8)]
    src = [rnd((rows, H, D), i, torch.bfloat16) for i in range(4)]
    for x, y in zip(views, src):
        x.copy_(y)
    cu = torch.tensor([0, 100, 300], dtype=torch.int32, device=DEV)
    o, lse = ftk.attn_fwd(*views[:3], cu, o=views[4])
    ref, rlse = ftk.attn_fwd(*src[:3], cu)
    assert torch.equal(o, ref) and torch.equal(lse, rlse)
    grads = ftk.attn_bwd(views[3], *views[:3], o, lse, cu, dq=views[5], dk=views[6], dv=views[7])
    for g, r in zip(grads, ftk.attn_bwd(src[3], *src[:3], ref, rlse, cu)):
        assert torch.equal(g, r)


@pytest.mark.parametrize("dtype,D", [(torch.float32, 16), (torch.bfloat16, 64)])
def test_many_short_sequences(dtype, D):
    rng = np.random.default_rng(3)
    lens = rng.integers(0, 4, 5000)
    q, k, v, cu = inputs(lens, 2, 1, D, dtype)
    o, lse = ftk.attn_fwd(q, k, v, cu)
    do = rnd(q.shape, 4, dtype)
    dq, dk, dv = ftk.attn_bwd(do, q, k, v, o, lse, cu)
    # sequences are independent: a sample of them, each in a batch of its own
    c = cu.tolist()
    for b in rng.integers(0, 5000, 60):
        s = slice(c[b], c[b + 1])
        n = c[b + 1] - c[b]
        if not n:
            continue
        one = torch.tensor([0, n], dtype=torch.int32, device=DEV)
        o1, l1 = ftk.attn_fwd(q[s], k[s], v[s], one)
        g1 = ftk.attn_bwd(do[s], q[s], k[s], v[s], o1, l1, one)
        for x, y in zip((o, lse.T, dq, dk, dv), (o1, l1.T, *g1)):
            assert torch.equal(x[s], y)


@pytest.mark.parametrize("dtype,D", [(torch.float32, 16), (torch.bfloat16, 64), (torch.bfloat16, 128)])
def test_guard_word_and_bad_boundaries(dtype, D):
    q, k, v, cu = inputs((50, 300), 4, 2, D, dtype)
    T = q.shape[0]
    do = rnd(q.shape, 4, dtype)
    o, lse = ftk.attn_fwd(q, k, v, cu)
    status = ftk.check_seqlens(cu, T)
    o2, lse2 = ftk.attn_fwd(q, k, v, cu, seqlens_status=status)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    g = ftk.attn_bwd(do, q, k, v, o, lse, cu)
    for a, b in zip(g, ftk.attn_bwd(do, q, k, v, o, lse, cu, seqlens_status=status)):
        assert torch.equal(a, b)
    for bad in ([0, 400, 350], [5, 300, 350], [0, 300, 100], [-7, 1 << 30, -(1 << 30)]):
        cub = torch.tensor(bad, dtype=torch.int32, device=DEV)
        status = ftk.check_seqlens(cub, T)
        o3 = torch.full_like(o, 7.0)
        l3 = torch.full_like(lse, 7.0)
        outs = [torch.full_like(t, 7.0) for t in (q, k, v)]
        ftk.attn_fwd(q, k, v, cub, o=o3, lse=l3, seqlens_status=status)
        ftk.attn_bwd(do, q, k, v, o, lse, cub, dq=outs[0], dk=outs[1], dv=outs[2],
                     seqlens_status=status)
        assert int(status.item()) != 0
        for t in (o3, l3, *outs):
            assert bool((t == 7).all())


@pytest.mark.parametrize("dtype,D", [(torch.float32, 32), (torch.bfloat16, 64), (torch.bfloat16, 128)])
def test_reproducible_on_streams_and_in_graphs(dtype, D):
    q, k, v, cu = inputs((300, 41, 700), 4, 2, D, dtype, fused=True)
    do = rnd(q.shape, 4, dtype)
    o, lse = ftk.attn_fwd(q, k, v, cu)
    g = ftk.attn_bwd(do, q, k, v, o, lse, cu)
    torch.cuda.synchronize()
    side = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for s in side:  # two calls at once
        with torch.cuda.stream(s):
            o2, l2 = ftk.attn_fwd(q, k, v, cu)
            got.append((o2, l2, *ftk.attn_bwd(do, q, k, v, o2, l2, cu)))
    torch.cuda.synchronize()
    for r in got:
        for a, b in zip(r, (o, lse, *g)):
            assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o3, l3 = ftk.attn_fwd(q, k, v, cu)
        g3 = ftk.attn_bwd(do, q, k, v, o3, l3, cu)
    for seed in (0, 77):  # replayed on new values in the same buffers, other lengths
        q.copy_(rnd(q.shape, seed, dtype))
        if seed:
            cu.copy_(torch.tensor([0, 11, 500, 1041], dtype=torch.int32, device=DEV))
        graph.replay()
        torch.cuda.synchronize()
        o4, l4 = ftk.attn_fwd(q, k, v, cu)
        for a, b in zip((o3, l3, *g3), (o4, l4, *ftk.attn_bwd(do, q, k, v, o4, l4, cu))):
            assert torch.equal(a, b)


def test_fused_gradient_buffer_and_no_lse():
    q, k, v, cu = inputs((90, 200), 4, 2, 64, torch.bfloat16, fused=True)
    o, lse = ftk.attn_fwd(q, k, v, cu)
    o2, none = ftk.attn_fwd(q, k, v, cu, save_lse=False)
    assert none is None and torch.equal(o, o2)
    do = rnd(q.shape, 4, q.dtype)
    g = ftk.attn_bwd(do, q, k, v, o, lse, cu)
    buf = torch.zeros(290, 8, 64, dtype=q.dtype, device=DEV)
    ftk.attn_bwd(do, q, k, v, o, lse, cu, dq=buf[:, :4], dk=buf[:, 4:6], dv=buf[:, 6:])
    assert torch.equal(buf, torch.cat(g, 1))


def test_empty_batch():
    x = torch.empty(0, 2, 64, dtype=torch.bfloat16, device=DEV)
    cu = torch.zeros(1, dtype=torch.int32, device=DEV)
    o, lse = ftk.attn_fwd(x, x, x, cu)
    assert o.shape == x.shape and lse.shape == (2, 0)
    assert all(t.shape == x.shape for t in ftk.attn_bwd(x, x, x, x, o, lse, cu))


def test_binding_refusals():
    q, k, v, cu = inputs((10,), 4, 2, 64, torch.bfloat16)
    with pytest.raises(ftk.FtkError):
        ftk.attn_fwd(q[:, :3], k, v, cu)  # 3 query heads over 2
    with pytest.raises(ftk.FtkError):
        ftk.attn_fwd(q, k, v, cu, o=q)
    with pytest.raises(ftk.FtkError):
        ftk.attn_fwd(q, k, v, cu, scale=-1.0)
    with pytest.raises(TypeError):
        ftk.attn_fwd(q.half(), k.half(), v.half(), cu)
    for args in ((q, k.float(), v, cu), (q, k, v[:5], cu), (q, k, v, cu.long()),
                 (q, k, v, cu.cpu()), (q[:, :, ::2], k[:, :, ::2], v[:, :, ::2], cu)):
        with pytest.raises(ValueError):
            ftk.attn_fwd(*args)
    o, lse = ftk.attn_fwd(q, k, v, cu)
    with pytest.raises(ValueError):
        ftk.attn_bwd(q, q, k, v, o, lse.T.contiguous(), cu)


# ------------------------------------------------------------------ rotation

def positions(T, seed, far=1):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return torch.randint(-3, 500 * far, (3, T), generator=g, device=DEV, dtype=torch.int32)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("Hq,Hkv,D", [(14, 2, 64), (32, 8, 128), (4, 2, 16), (3, 1, 80), (2, 2, 6),
                                      (1, 0, 2), (0, 3, 96), (2, 1, 512), (40, 40, 256)])
def test_mrope(Hq, Hkv, D, dtype):
    theta = 1e6
    freq = [theta ** (-2 * i / D) for i in range(D // 2)]
    for T, far in ((1, 1), (7, 1), (333, 1000)):
        q = rnd((T, Hq, D), 1, dtype) if Hq else None
        k = rnd((T, Hkv, D), 2, dtype) if Hkv else None
        pos = positions(T, 3, far)
        axis = [i % 3 for i in range(D // 2)]
        for fn, sign in ((ftk.qk_mrope_fwd, 1.0), (ftk.qk_mrope_bwd, -1.0)):
            outs = fn(q, k, pos, axis, theta=theta)
            for x, y in zip((q, k), outs):
                if x is not None:
                    within(f"{T}", y, *A.qk_mrope(x, pos, axis, freq, sign, CODE[dtype]))
            table = fn(q, k, pos, axis, inv_freq=freq)
            twin = fn(q.clone() if Hq else None, k.clone() if Hkv else None, pos, axis, theta=theta)
            for x, y, z in zip(outs, table, twin):
                assert x is None or (torch.equal(x, y) and torch.equal(x, z))


def test_mrope_in_place_strided_and_equal_axes():
    T, Hq, Hkv, D, theta = 100, 6, 2, 64, 1e6
    x = rnd((T, Hq + 2 * Hkv, D), 1, torch.bfloat16)
    v = x[:, Hq + Hkv:].clone()
    pos = torch.arange(T, dtype=torch.int32, device=DEV).expand(3, T)  # one row, stride 0
    axis = ftk.mrope_axis_of((8, 12, 12))
    with pytest.raises(ftk.FtkError):
        ftk.qk_mrope_fwd(x[:, :Hq], x[:, Hq:Hq + Hkv], pos, axis, theta=theta)
    pos = pos.contiguous()
    q2, k2 = x[:, :Hq].clone(), x[:, Hq:Hq + Hkv].clone()
    ftk.qk_rope_fwd(q2, k2, torch.tensor([0, T], dtype=torch.int32, device=DEV), theta)
    q, k = x[:, :Hq], x[:, Hq:Hq + Hkv]
    ftk.qk_mrope_fwd(q, k, pos, axis, theta=theta, q_out=q, k_out=k)
    # the same angles as the one-axis rotation, and at most one rounding apart
    for a, b in ((q, q2), (k, k2)):
        assert bool(((a.float() - b.float()).abs() <= 2.0 ** -7 * b.float().abs() + 2e-6).all())
    assert torch.equal(x[:, Hq + Hkv:], v)
    wide = torch.zeros(3, T + 5, dtype=torch.int32, device=DEV)
    wide[:, :T] = pos
    a, b = ftk.qk_mrope_fwd(q, k, wide[:, :T], axis, theta=theta), ftk.qk_mrope_fwd(
        q, k, pos, axis, theta=theta)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    # off a 16-byte boundary: the element-wise form, the same bits
    off = torch.empty(T * Hq * D + 1, dtype=q.dtype, device=DEV)[1:].view(T, Hq, D)
    off.copy_(q)
    c = ftk.qk_mrope_fwd(off, k.contiguous(), pos, axis, theta=theta)
    assert torch.equal(c[0], b[0]) and torch.equal(c[1], b[1])


def test_mrope_empty_and_graph():
    e = torch.empty(0, 2, 64, dtype=torch.bfloat16, device=DEV)
    pos = torch.empty(3, 0, dtype=torch.int32, device=DEV)
    axis = ftk.mrope_axis_of((8, 12, 12))
    assert ftk.qk_mrope_fwd(e, e, pos, axis, theta=1e4)[0].shape == e.shape
    q, k, pos = rnd((50, 4, 64), 1, torch.bfloat16), rnd((50, 2, 64), 2, torch.bfloat16), positions(50, 3)
    graph = torch.cuda.CUDAGraph()
    ftk.qk_mrope_fwd(q, k, pos, axis, theta=1e4)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        a = ftk.qk_mrope_fwd(q, k, pos, axis, theta=1e4)
    pos.copy_(positions(50, 4))
    graph.replay()
    b = ftk.qk_mrope_fwd(q, k, pos, axis, theta=1e4)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


# ------------------------------------------------------------------ together

def test_a_layers_attention_block_with_its_gradients():
    """norm -> rotation by three axes -> attention, forward and backward through
    autograd, in bf16, against the same block in 64 bits.  Every stored tensor
    of the chain rounds once (2^-8 each: q, k, o and back), so the result is
    compared in the 2-norm against the sum of those roundings."""
    lens, Hq, Hkv, D, theta = (37, 1, 200, 90), 4, 2, 64, 1e6
    q0, k0, v0, cu = inputs(lens, Hq, Hkv, D, torch.bfloat16)
    T = q0.shape[0]
    pos, axis = positions(T, 5), ftk.mrope_axis_of((8, 12, 12))
    do = rnd(q0.shape, 6, q0.dtype)
    leaves = [t.clone().requires_grad_(True) for t in (q0, k0, v0)]
    q, k = autograd.qk_mrope(leaves[0], leaves[1], pos, axis, theta)
    o = autograd.attention(q, k, leaves[2], cu)
    o.backward(do)

    ref = [t.double().requires_grad_(True) for t in (q0, k0, v0)]
    f = torch.tensor([theta ** (-2 * i / D) for i in range(D // 2)], dtype=torch.float64, device=DEV)
    phi = pos.double()[torch.as_tensor(axis, device=DEV).long()].T * f
    c, s = phi.cos()[:, None], phi.sin()[:, None]
    turn = lambda x: torch.cat([x[..., :32] * c - x[..., 32:] * s,  # noqa: E731
                                x[..., 32:] * c + x[..., :32] * s], -1)
    qr, kr = turn(ref[0]), turn(ref[1])
    out, a = [], 0
    for n in lens:
        z = torch.einsum("ihd,jhd->hij", qr[a:a + n], kr[a:a + n].repeat_interleave(2, 1)) / 8
        z = z.masked_fill(torch.ones(n, n, dtype=torch.bool, device=DEV).triu(1), -math.inf)
        out.append(torch.einsum("hij,jhd->ihd", z.softmax(-1), ref[2][a:a + n].repeat_interleave(2, 1)))
        a += n
    ro = torch.cat(out)
    ro.backward(do.double())
    far = lambda x, y: float((x.detach().double() - y.detach()).norm() / y.detach().norm())  # noqa: E731
    # o: q, k rounded (2^-8 of scores of size ~sqrt(D) / 8 = 1, twice), p and o: 4 roundings;
    # the gradients pass dp, ds and the turned-back rounding as well: 8
    assert far(o, ro) < 4 * 2.0 ** -8
    for x, y in zip(leaves, ref):
        assert far(x.grad, y.grad) < 8 * 2.0 ** -8


def test_autograd_equals_the_direct_calls():
    q0, k0, v0, cu = inputs((60, 70), 4, 2, 64, torch.bfloat16, fused=True)
    do = rnd((130, 4, 64), 6, q0.dtype)
    for causal in (True, False):
        leaves = [t.clone().requires_grad_(True) for t in (q0, k0, v0)]
        autograd.attention(*leaves, cu, 0.2, causal).backward(do)
        o, lse = ftk.attn_fwd(q0, k0, v0, cu, scale=0.2, causal=causal)
        for a, b in zip(leaves, ftk.attn_bwd(do, q0, k0, v0, o, lse, cu, scale=0.2, causal=causal)):
            assert torch.equal(a.grad, b)


def test_autograd_on_a_padded_batch():
    """Rows of no sequence: whatever stands there, zero output and gradients."""
    q0, k0, v0, cu = inputs((60, 70), 4, 2, 64, torch.bfloat16, lead=3, tail=50)
    pad = torch.ones(183, dtype=torch.bool, device=DEV)
    pad[3:133] = False
    do = rnd(q0.shape, 6, q0.dtype)
    for t in (q0, k0, v0, do):
        t[pad] = math.nan
    leaves = [t.clone().requires_grad_(True) for t in (q0, k0, v0)]
    o = autograd.attention(*leaves, cu)
    o.backward(do)
    assert bool((o[pad] == 0).all())
    one = [t[3:133].clone().requires_grad_(True) for t in (q0, k0, v0)]
    p = autograd.attention(*one, cu - 3)
    p.backward(do[3:133])
    assert torch.equal(o[3:133], p)
    for a, b in zip(leaves, one):
        assert bool((a.grad[pad] == 0).all())
        assert torch.equal(a.grad[3:133], b.grad)


def test_autograd_captured_with_its_gradients():
    q0, k0, v0, cu = inputs((60, 70), 4, 2, 64, torch.bfloat16)
    pos, axis = positions(130, 5), ftk.mrope_axis_of((8, 12, 12))
    do = rnd(q0.shape, 6, q0.dtype)
    leaves = [t.clone().requires_grad_(True) for t in (q0, k0, v0)]

    def step():
        q, k = autograd.qk_mrope(leaves[0], leaves[1], pos, axis, 1e6)
        o = autograd.attention(q, k, leaves[2], cu)
        return (o.detach(), *torch.autograd.grad(o, leaves, do))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for seed in (11, 12):
        with torch.no_grad():
            for i, t in enumerate(leaves):
                t.copy_(rnd(t.shape, seed + 10 * i, t.dtype))
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, step()):
            assert torch.equal(a, b)


def test_second_derivatives_are_refused():
    q, k, v, cu = inputs((20, 30), 4, 2, 64, torch.bfloat16)
    pos, axis = positions(50, 5), ftk.mrope_axis_of((8, 12, 12))
    q, k = q.requires_grad_(True), k.requires_grad_(True)
    for out in (autograd.attention(q, k, v, cu), autograd.qk_mrope(q, k, pos, axis, 1e6)[0]):
        (g,) = torch.autograd.grad(out.float().square().sum(), q, create_graph=True)
        with pytest.raises(RuntimeError):
            torch.autograd.grad(g.float().sum(), q)


def test_expanded_heads_and_tokens_are_refused():
    """Broadcast views have no row per token and head to read."""
    q, k, v, cu = inputs((20, 30), 4, 2, 64, torch.bfloat16)
    with pytest.raises(ValueError):
        ftk.attn_fwd(q, k[:, :1].expand(50, 2, 64), v, cu)
    with pytest.raises((ValueError, ftk.FtkError)):
        ftk.attn_fwd(q, k[:1].expand(50, 2, 64), v, cu)


# ------------------------------------------------------------------ rules by size

@pytest.mark.parametrize("Hq,Hkv,D,lens", [
    # 32 key tiles or more of 16 key heads: a group's heads stay in one CTA
    (32, 16, 64, (1500, 700, 232, 100)), (32, 16, 128, (1500, 700, 232, 100)),
    # some 50 tiles of 2 key heads: seven heads dealt to four CTAs, unevenly
    (14, 2, 64, (900, 1, 700) * 4), (14, 2, 128, (900, 1, 700) * 4)])
def test_shared_heads_by_the_number_of_key_tiles(Hq, Hkv, D, lens):
    check(*inputs(lens, Hq, Hkv, D, torch.bfloat16, fused=True), True)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("B", [2, 127, 128, 129])
def test_batches_around_the_length_order(B, D):
    """Up to 128 sequences are taken by length, more by position; empty ones,
    equal ones and a long one among them."""
    lens = np.random.default_rng(B).integers(0, 40, B)
    lens[B // 2] = 600
    lens[-1] = 0 if B > 2 else 17
    check(*inputs(tuple(int(n) for n in lens), 4, 2, D, torch.bfloat16, lead=5, tail=9), True)
