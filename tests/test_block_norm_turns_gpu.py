"""The joint where a row group works on many rows, several at a time, with later rows on
their way: rows do not reach one another, and outputs may take the place of inputs; wide
rows that are not aligned."""
import pytest
import torch

from test_block_norm_gpu import DT, EPS, case, check_bwd, check_fwd, ftk

pytestmark = pytest.mark.gpu
# (T, H): every group has several turns, the last one short.  One warp a row, several rows a
# CTA, 16 and 20 warps, two and four packets, single columns by four and eight, any length
TURNS = [(40000, 64), (5000, 896), (1300, 4096), (1300, 5120), (900, 8200), (700, 12000),
         (40000, 24), (30001, 61), (1300, 1001), (900, 4993), (2600, 5131)]


def both(c, f, h=None, y=None, dx=None, dres=None):
    kw = dict(**f, res_scale=0.7, x_scale=0.4, p=0.25, seed=1)
    out = ftk().rmsnorm_block_fwd(c["x"], c["res"], c["w"], EPS, **kw, h=h, y=y)
    return out, kw


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("T, H", TURNS)
def test_rows_that_share_a_turn(dtype, T, H):
    c, f = case(T, H, dtype)
    g = torch.Generator(device="cuda").manual_seed(7)
    hit = torch.rand(T, generator=g, device="cuda") < 0.1  # with any stride, next to good ones
    value = torch.where(torch.rand(T, generator=g, device="cuda") < 0.5, float("nan"), float("inf"))
    bad = dict(c)
    for n in ("x", "res", "dy", "dh"):
        bad[n] = torch.where(hit[:, None], value[:, None].to(c[n].dtype), c[n])
    rows = []
    for v in (c, bad):
        (h, y, r, r1), kw = both(v, f)
        dx, dres, *_, dt = ftk().rmsnorm_block_bwd(v["dy"], v["dh"], v["x"], h, v["w"], r, r1, **kw)
        rows.append((h, y, r, r1, dx, dres, dt))
    assert 0 < int(hit.sum()) < T
    for a, b in zip(*rows):
        assert torch.equal(a[~hit], b[~hit])
        assert not torch.isfinite(b[hit].float()).all()


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("T, H", TURNS)
def test_in_place_while_later_rows_are_on_their_way(dtype, T, H):
    c, f = case(T, H, dtype)
    (h, y, r, r1), kw = both(c, f)
    for n in ("res", "x"):
        own = {**c, n: c[n].clone()}
        out, _ = both(own, f, h=own[n])
        assert out[0].data_ptr() == own[n].data_ptr()
        for a, b in zip((h, y, r, r1), out):
            assert torch.equal(a, b), n
    args = (c["x"], h, c["w"], r, r1)
    ref = ftk().rmsnorm_block_bwd(c["dy"], c["dh"], *args, **kw)
    for swap in (False, True):
        dy, dh = c["dy"].clone(), c["dh"].clone()
        got = ftk().rmsnorm_block_bwd(dy, dh, *args, **kw, dx=dh if swap else dy,
                                      dres=dy if swap else dh)
        for a, b in zip(ref, got):
            assert torch.equal(a, b), swap


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("H", [8192, 5131])
@pytest.mark.parametrize("shift", [0, 1, 8])
def test_wide_rows_of_views(dtype, H, shift):
    # 8,192 columns from an odd offset on are single ones, and too many for the register kernels
    T = 330
    c, f = case(T, H, dtype)
    kw = dict(**f, res_scale=0.7, x_scale=0.4, p=0.25, seed=1)
    wide = {n: torch.full((T, H + 40), 5.0, device="cuda", dtype=DT[dtype])
            for n in ("x", "res", "h", "y", "dy", "dh", "dx", "dres")}
    v = {n: t[:, shift:shift + H] for n, t in wide.items()}
    for n in ("x", "res", "dy", "dh"):
        v[n].copy_(c[n])
    out = ftk().rmsnorm_block_fwd(v["x"], v["res"], c["w"], EPS, **kw, h=v["h"], y=v["y"])
    check_fwd(c, f, 0.7, 0.4, 0.25, out)
    grads = ftk().rmsnorm_block_bwd(v["dy"], v["dh"], v["x"], v["h"], c["w"], *out[2:], **kw,
                                    dx=v["dx"], dres=v["dres"])
    check_bwd(c, f, 0.7, 0.4, 0.25, out[0], out[2], out[3], grads)
    for t in wide.values():
        assert (t[:, :shift] == 5).all() and (t[:, shift + H:] == 5).all()
