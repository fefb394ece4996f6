"""The joint of a block's output with the residual stream on the GPU, forward and
backward, against the 64-bit oracle and the bars that it derives."""
import itertools

import pytest
import torch

from oracle import residual as R

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
EPS = 1e-5
SIZES = [(1, 1), (1, 8), (3, 7), (64, 64), (5, 257), (33, 896), (9, 1001), (70, 2048), (4, 4096),
         (7, 5120), (2, 8200), (3, 16384), (2, 20000), (2, 5003), (3, 5131), (2, 20487), (1000, 24),
         (2500, 128), (650, 640), (613, 321), (331, 5120), (400, 5131), (500, 6000), (350, 12000), (320, 18000),
         (400, 9600), (1300, 4993), (700, 2500), (310, 4096)]


def ftk():
    from fine_tuning_gb300 import ftk as f
    return f


def case(T, H, dtype, post=True, gate=True, tok=True, seed=0, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda")
    dt = DT[dtype]
    c = {"x": (std * rand(T, H)).to(dt), "res": (2 * rand(T, H)).to(dt),
         "w": (1 + 0.1 * rand(H)).to(dt), "dy": rand(T, H).to(dt), "dh": rand(T, H).to(dt)}
    f = {"w_post": (1 + 0.1 * rand(H)).to(dt) if post else None,
         "gate": (0.5 + 0.3 * rand(H)).to(dt) if gate else None,
         "gate_tok": torch.sigmoid(rand(T)) if tok else None}
    return c, f


def close(name, got, ref, bar):
    if ref is None:
        assert got is None, name
        return
    bad = ~((got.cpu().double() - ref).abs() <= bar)
    assert not bad.any(), (name, int(bad.sum()), tuple(got.shape))


def check_fwd(c, f, a, b, p, out, seed=1, offset=0, eps=EPS):
    h, y, r, r1 = out
    keep = R.keep_mask(*h.shape, p, seed, offset) if p else None
    (h0, r10), (bh, b1) = R.block_fwd(c["x"], c["res"], c["w"], eps, **f, res_scale=a, x_scale=b,
                                      keep=keep, p=p)
    (y0, r0), (by, br) = R.block_y(h, c["w"], eps)
    for n, g, v, t in (("h", h, h0, bh), ("rstd_post", r1, r10, b1), ("y", y, y0, by),
                       ("rstd", r, r0, br)):
        close(n, g, v, t)


NAMES = ("dx", "dres", "dw", "dw_post", "dgate", "dgate_tok")


def check_bwd(c, f, a, b, p, h, r, r1, out, seed=1, offset=0):
    keep = R.keep_mask(*h.shape, p, seed, offset) if p else None
    ref, bar = R.block_bwd(c["dy"], c["dh"], c["x"], h, c["w"], r, r1, **f, res_scale=a, x_scale=b,
                           keep=keep, p=p)
    for n, g, v, t in zip(NAMES, out, ref, bar):
        close(n, g, v, t)


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("T, H", SIZES)
@pytest.mark.parametrize("p", [0.0, 0.25])
def test_everything_at_once(dtype, T, H, p):
    c, f = case(T, H, dtype)
    kw = dict(res_scale=0.7, x_scale=0.4, p=p, seed=1)
    out = h, y, r, r1 = ftk().rmsnorm_block_fwd(c["x"], c["res"], c["w"], EPS, **f, **kw)
    check_fwd(c, f, 0.7, 0.4, p, out)
    args = (c["dy"], c["dh"], c["x"], h, c["w"], r, r1)
    grads = ftk().rmsnorm_block_bwd(*args, **f, **kw)
    check_bwd(c, f, 0.7, 0.4, p, h, r, r1, grads)
    for g, again in zip(grads, ftk().rmsnorm_block_bwd(*args, **f, **kw)):
        assert torch.equal(g, again)


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("post, gate, tok", list(itertools.product([False, True], repeat=3)))
@pytest.mark.parametrize("H", [96, 99, 2056])
def test_factors_left_out(dtype, post, gate, tok, H):
    for p in (0.0, 0.5):
        c, f = case(21, H, dtype, post, gate, tok)
        out = h, y, r, r1 = ftk().rmsnorm_block_fwd(c["x"], c["res"], c["w"], EPS, **f, p=p, seed=1)
        check_fwd(c, f, 1.0, 1.0, p, out)
        grads = ftk().rmsnorm_block_bwd(c["dy"], c["dh"], c["x"], h, c["w"], r, r1, **f, p=p, seed=1)
        check_bwd(c, f, 1.0, 1.0, p, h, r, r1, grads)


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("H", [64, 61])
def test_without_factors_it_is_the_residual_norm(dtype, H):
    c, _ = case(50, H, dtype)
    h, y, r, _ = ftk().rmsnorm_block_fwd(c["x"], c["res"], c["w"], EPS)
    h0, y0, r0 = ftk().rmsnorm_add_fwd(c["x"], c["res"], c["w"], EPS)
    assert torch.equal(h, h0)
    u = torch.finfo(DT[dtype]).eps + 2 * R.rstd_error(H)  # two roundings, two sums of squares
    assert ((y.double() - y0.double()).abs() <= u * y0.double().abs()).all()


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("H", [128, 127, 4096])
def test_views_and_in_place(dtype, H):
    T, p = 11, 0.25
    c, f = case(T, H, dtype)
    kw = dict(**f, p=p, seed=1)
    base = ftk().rmsnorm_block_fwd(c["x"], c["res"], c["w"], EPS, **kw)
    for a in (0, 1, 8):
        wide = {n: torch.full((T, H + 40), 5.0, device="cuda", dtype=DT[dtype])
                for n in ("x", "res", "h", "y", "dy", "dh", "dx", "dres")}
        v = {n: t[:, a:a + H] for n, t in wide.items()}
        for n in ("x", "res", "dy", "dh"):
            v[n].copy_(c[n])
        out = ftk().rmsnorm_block_fwd(v["x"], v["res"], c["w"], EPS, **kw, h=v["h"], y=v["y"])
        check_fwd(c, f, 1.0, 1.0, p, out)
        grads = ftk().rmsnorm_block_bwd(v["dy"], v["dh"], v["x"], v["h"], c["w"], *out[2:], **kw,
                                        dx=v["dx"], dres=v["dres"])
        check_bwd(c, f, 1.0, 1.0, p, out[0], out[2], out[3], grads)
        for t in wide.values():
            assert (t[:, :a] == 5).all() and (t[:, a + H:] == 5).all()
    # h in the place of the stream or of the block's output
    for n in ("res", "x"):
        own = {m: c[m].clone() for m in ("x", "res")}
        out = ftk().rmsnorm_block_fwd(own["x"], own["res"], c["w"], EPS, **kw, h=own[n])
        for g, b in zip(out, base):
            assert torch.equal(g, b)
        assert out[0].data_ptr() == own[n].data_ptr()
    # gradients in the place of those that arrive
    h, _, r, r1 = base
    ref = ftk().rmsnorm_block_bwd(c["dy"], c["dh"], c["x"], h, c["w"], r, r1, **kw)
    for swap in (False, True):
        dy, dh = c["dy"].clone(), c["dh"].clone()
        got = ftk().rmsnorm_block_bwd(dy, dh, c["x"], h, c["w"], r, r1, **kw,
                                      dx=dh if swap else dy, dres=dy if swap else dh)
        for g, b in zip(got, ref):
            assert torch.equal(g, b)


@pytest.mark.parametrize("dtype", DT)
def test_halves_of_one_buffer_and_weights_anywhere(dtype):
    T, H = 200, 128
    c, f = case(T, H, dtype)
    pool = torch.zeros(4 * H + 8, device="cuda", dtype=DT[dtype])
    for shift in (0, 1):
        both = torch.cat([c["x"], c["res"]], 1)
        w, wp, g = (pool[shift + i * (H + 1) * (1 if shift else 0) + i * H * (0 if shift else 1):][:H]
                    for i in range(3))
        w.copy_(c["w"]), wp.copy_(f["w_post"]), g.copy_(f["gate"])
        kw = dict(w_post=wp, gate=g, gate_tok=f["gate_tok"], p=0.25, seed=1)
        out = torch.empty(T, 2 * H, device="cuda", dtype=DT[dtype])
        got = ftk().rmsnorm_block_fwd(both[:, :H], both[:, H:], w, EPS, **kw, h=out[:, :H],
                                      y=out[:, H:])
        check_fwd(c, f, 1.0, 1.0, 0.25, got)
        grads = torch.cat([c["dy"], c["dh"]], 1)
        res = ftk().rmsnorm_block_bwd(grads[:, :H], grads[:, H:], both[:, :H], out[:, :H], w, got[2],
                                      got[3], **kw, dx=grads[:, H:], dres=grads[:, :H])
        check_bwd(c, f, 1.0, 1.0, 0.25, got[0], got[2], got[3], res)


def test_refusals():
    from fine_tuning_gb300.ftk import FtkError
    c, f = case(40, 64, "bf16")
    fwd = lambda **kw: ftk().rmsnorm_block_fwd(c["x"], c["res"], c["w"], EPS, **{**f, **kw})
    h, y, r, r1 = fwd()
    assert fwd(save_rstd=False)[2:] == (None, None)
    for kw in (dict(y=c["x"]), dict(y=c["res"]), dict(h=h, y=h), dict(p=1.5), dict(x_scale=float("nan"))):
        with pytest.raises(FtkError):
            fwd(**kw)
    for kw in (dict(w_post=c["w"][:32]), dict(gate=c["w"].float()), dict(gate_tok=f["gate_tok"].half()),
               dict(h=h[:3]), dict(seed=-1), dict(step=torch.zeros(1, device="cuda"))):
        with pytest.raises(ValueError):
            fwd(**kw)
    bwd = lambda **kw: ftk().rmsnorm_block_bwd(c["dy"], c["dh"], c["x"], h, c["w"], r,
                                               **{"rstd_post": r1, **f, **kw})
    for kw in (dict(dx=c["x"]), dict(dx=h), dict(dx=c["dy"], dres=c["dy"]),
               dict(workspace=torch.empty(1024, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(FtkError):
            bwd(**kw)
    for kw in (dict(rstd_post=None), dict(rstd_post=r1[:3]), dict(dres=y[:, :8])):
        with pytest.raises(ValueError):
            bwd(**kw)
    with pytest.raises(TypeError):
        ftk().dropout_fwd(c["x"].half(), 0.1, 1)


@pytest.mark.parametrize("H", [64, 61])
def test_mask_is_the_dropouts(H):
    T = 40
    x = torch.ones(T, H, device="cuda")
    res = torch.zeros(T, H, device="cuda")
    step = torch.tensor([2], device="cuda")
    h = ftk().rmsnorm_block_fwd(x, res, x[0], EPS, p=0.3, seed=77, offset=9, step=step)[0]
    assert torch.equal(h, ftk().dropout_fwd(x, 0.3, 77, 9, step))


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("H", [64, 61, 5131])
def test_dropped_infinities_reach_nothing(dtype, H):
    T, p = 9, 0.5
    c, f = case(T, H, dtype, post=False)
    kw = dict(**f, p=p, seed=1)
    keep = R.keep_mask(T, H, p, 1).cuda()
    bad = c["x"].clone()
    bad[~keep] = float("inf")
    bad[:, ::2][~keep[:, ::2]] = float("nan")
    out = ftk().rmsnorm_block_fwd(c["x"], c["res"], c["w"], EPS, **kw)
    got = ftk().rmsnorm_block_fwd(bad, c["res"], c["w"], EPS, **kw)
    for a, b in zip(out[:3], got[:3]):
        assert torch.equal(a, b)
    h, _, r, _ = out
    for a, b in zip(ftk().rmsnorm_block_bwd(c["dy"], c["dh"], c["x"], h, c["w"], r, **kw),
                    ftk().rmsnorm_block_bwd(c["dy"], c["dh"], bad, h, c["w"], r, **kw)):
        assert (a is None and b is None) or torch.equal(a, b)


@pytest.mark.parametrize("H", [64, 61])
def test_all_dropped_or_gated_off(H):
    c, f = case(13, H, "bf16")
    out = ftk().rmsnorm_block_fwd(c["x"], c["res"], c["w"], EPS, **f, p=1.0)
    assert torch.equal(out[0], c["res"])
    dx, dres, _, dwp, dg, dt = ftk().rmsnorm_block_bwd(c["dy"], c["dh"], c["x"], *out[:1], c["w"],
                                                       *out[2:], **f, p=1.0)
    for t in (dx, dwp, dg, dt):
        assert (t == 0).all()
    # a token's gate of 0 leaves its stream alone, and still has a gradient
    f["gate_tok"] = torch.zeros(13, device="cuda")
    out = h, y, r, r1 = ftk().rmsnorm_block_fwd(c["x"], c["res"], c["w"], EPS, **f)
    assert torch.equal(h, c["res"])
    grads = ftk().rmsnorm_block_bwd(c["dy"], c["dh"], c["x"], h, c["w"], r, r1, **f)
    check_bwd(c, f, 1.0, 1.0, 0.0, h, r, r1, grads)
    assert (grads[0] == 0).all() and (grads[5] != 0).any()


@pytest.mark.parametrize("H", [64, 61, 1024])
@pytest.mark.parametrize("std", [0.0, 1e-18, 1e15])
def test_rows_near_zero_and_large(H, std):
    # r1 reaches 1 / sqrt(eps) = 1e9 and r1^3 would overflow; with std = 1e15 it is 1e-15
    c, f = case(6, H, "f32", std=std)
    out = h, y, r, r1 = ftk().rmsnorm_block_fwd(c["x"], c["res"], c["w"], 1e-18, **f, p=0.25, seed=1)
    check_fwd(c, f, 1.0, 1.0, 0.25, out, eps=1e-18)
    grads = ftk().rmsnorm_block_bwd(c["dy"], c["dh"], c["x"], h, c["w"], r, r1, **f, p=0.25, seed=1)
    check_bwd(c, f, 1.0, 1.0, 0.25, h, r, r1, grads)


def test_rows_do_not_reach_one_another():
    c, f = case(24, 256, "bf16")
    kw = dict(**f, p=0.25, seed=1)
    h, y, r, r1 = ftk().rmsnorm_block_fwd(c["x"], c["res"], c["w"], EPS, **kw)
    dx, dres = ftk().rmsnorm_block_bwd(c["dy"], c["dh"], c["x"], h, c["w"], r, r1, **kw)[:2]
    bad = {n: c[n].clone() for n in ("x", "res", "dy", "dh")}
    for t in bad.values():
        t[5], t[17] = float("nan"), float("inf")
    h2, y2, r2, r12 = ftk().rmsnorm_block_fwd(bad["x"], bad["res"], c["w"], EPS, **kw)
    dx2, dres2 = ftk().rmsnorm_block_bwd(bad["dy"], bad["dh"], bad["x"], h2, c["w"], r2, r12, **kw)[:2]
    rest = [i for i in range(24) if i not in (5, 17)]
    for a, b in ((h, h2), (y, y2), (r, r2), (r1, r12), (dx, dx2), (dres, dres2)):
        assert torch.equal(a[rest], b[rest])


def test_empty_batch():
    c, f = case(0, 64, "bf16")
    h, y, r, r1 = ftk().rmsnorm_block_fwd(c["x"], c["res"], c["w"], EPS, **f)
    grads = ftk().rmsnorm_block_bwd(c["dy"], c["dh"], c["x"], h, c["w"], r, r1, **f)
    assert h.shape == y.shape == grads[0].shape == (0, 64) and grads[5].shape == (0,)
    for g in grads[2:5]:
        assert g.shape == (64,) and (g == 0).all()


def test_rows_past_31_bits():
    T, H = 2 ** 20 + 5, 2056  # 2.16e9 elements
    x = torch.ones(T, H, device="cuda", dtype=torch.bfloat16)
    c, f = case(6, H, "bf16", tok=False)
    res, dy, dh = (torch.zeros_like(x) for _ in range(3))
    x[-6:], res[-6:] = c["x"], c["res"]
    h, y, r, r1 = ftk().rmsnorm_block_fwd(x, res, c["w"], EPS, **f)
    check_fwd(c, f, 1.0, 1.0, 0.0, (h[-6:], y[-6:], r[-6:], r1[-6:]))
    dy[-6:], dh[-6:] = c["dy"], c["dh"]
    grads = ftk().rmsnorm_block_bwd(dy, dh, x, h, c["w"], r, r1, **f, dx=dy, dres=dh)
    check_bwd(c, f, 1.0, 1.0, 0.0, h[-6:], r[-6:], r1[-6:],
              (grads[0][-6:], grads[1][-6:], *grads[2:]))  # the other rows' gradients are zeros


@pytest.mark.parametrize("dtype", DT)
def test_autograd(dtype):
    from fine_tuning_gb300 import autograd
    c, f = case(30, 64, dtype)
    leaf = {n: v.clone().requires_grad_() for n, v in {**c, **f}.items() if n not in ("dy", "dh")}
    step = torch.ones(1, dtype=torch.int64, device="cuda")
    h, y = autograd.rmsnorm_block(leaf["x"], leaf["res"], leaf["w"], EPS, leaf["w_post"], leaf["gate"],
                                  leaf["gate_tok"], 0.7, 0.4, 0.25, 1, 2, step)
    torch.autograd.backward([h, y], [c["dh"], c["dy"]])
    out = ftk().rmsnorm_block_fwd(c["x"], c["res"], c["w"], EPS, **f, res_scale=0.7, x_scale=0.4,
                                  p=0.25, seed=1, offset=3)
    ref = ftk().rmsnorm_block_bwd(c["dy"], c["dh"], c["x"], out[0], c["w"], *out[2:], **f,
                                  res_scale=0.7, x_scale=0.4, p=0.25, seed=1, offset=3)
    for n, g in zip(("x", "res", "w", "w_post", "gate", "gate_tok"), ref):
        assert torch.equal(leaf[n].grad, g.to(leaf[n].dtype)), n
    # one output alone
    x = leaf["x"].detach().requires_grad_()
    autograd.rmsnorm_block(x, leaf["res"].detach(), leaf["w"].detach(), EPS)[1].sum().backward()
    assert torch.isfinite(x.grad).all()
