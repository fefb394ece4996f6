"""The joint's backward for rows near zero without an eps: r1 or r2 is 2^62, whose square
times a gradient of 2^10 does not fit fp32, while every gradient does."""
import pytest
import torch

from oracle import residual as R
from test_block_norm_gpu import check_bwd, check_fwd, ftk

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
SMALL, LARGE = 2.0 ** -62, 2.0 ** 10


def case(T, H, dtype, where):
    """where "stream": res and what x brings to it are near zero; "block": x is."""
    g = torch.Generator(device="cuda").manual_seed(H)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda")
    dt = DT[dtype]
    x, res = rand(T, H), rand(T, H)
    f = {"w_post": (1 + 0.1 * rand(H)).to(dt), "gate": (0.5 + 0.3 * rand(H)).to(dt),
         "gate_tok": torch.sigmoid(rand(T))}
    # gradients that lie along the rows, so that the sums over a row do not cancel
    c = {"x": (x * (SMALL if where == "block" else 1)).to(dt),
         "res": (res * (SMALL if where == "stream" else 1)).to(dt),
         "w": (1 + 0.1 * rand(H)).to(dt), "dy": (LARGE * (res + 0.5 * rand(T, H))).to(dt),
         "dh": (LARGE * (x + 0.5 * rand(T, H))).to(dt)}
    return c, f, SMALL / 4 if where == "stream" else 0.4


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("where", ["stream", "block"])
# one warp a row, several, 20 warps, two and four packets, single columns by four and eight,
# and the kernel for any length
@pytest.mark.parametrize("H", [64, 896, 4096, 5120, 8200, 12000, 24, 61, 1001, 4993, 5131])
@pytest.mark.parametrize("p", [0.0, 0.25])
def test_gradients_that_fit(dtype, where, H, p):
    c, f, b = case(7, H, dtype, where)
    kw = dict(res_scale=0.7, x_scale=b, p=p, seed=1)
    out = h, y, r, r1 = ftk().rmsnorm_block_fwd(c["x"], c["res"], c["w"], 0.0, **f, **kw)
    check_fwd(c, f, 0.7, b, p, out, eps=0.0)
    grads = ftk().rmsnorm_block_bwd(c["dy"], c["dh"], c["x"], h, c["w"], r, r1, **f, **kw)
    check_bwd(c, f, 0.7, b, p, h, r, r1, grads)


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("H", [896, 61])
def test_without_the_blocks_norm(dtype, H):
    c, f, b = case(7, H, dtype, "stream")
    f["w_post"] = None
    h, y, r, _ = ftk().rmsnorm_block_fwd(c["x"], c["res"], c["w"], 0.0, **f, x_scale=b)
    grads = ftk().rmsnorm_block_bwd(c["dy"], c["dh"], c["x"], h, c["w"], r, **f, x_scale=b)
    check_bwd(c, f, 1.0, b, 0.0, h, r, None, grads)
