"""Dropout on the GPU against the 64-bit oracle: the mask exactly, the kept values
to the roundings that the oracle counts."""
import pytest
import torch

from oracle import residual as R

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
SEED = 0xFEDCBA9876543210


def ftk():
    from fine_tuning_gb300 import ftk as f
    return f


def values(T, H, dtype, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(T, H, generator=g, device="cuda").to(dtype)


def check(y, ref):
    ref, bar = ref
    bad = ~((y.cpu().double() - ref).abs() <= bar)
    assert not bad.any(), (int(bad.sum()), y.shape)
    assert torch.equal(y.cpu().double() == 0, ref == 0)


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("T, H", [(1, 1), (1, 8), (3, 7), (5, 16), (33, 64), (2, 257), (17, 1001),
                                  (64, 896), (3, 4104), (1, 70000), (4099, 24), (5, 12), (9, 20),
                                  (20000, 40), (3001, 2048)])
@pytest.mark.parametrize("p", [0.0, 0.1, 0.5, 1.0])
def test_forward_and_backward(dtype, T, H, p):
    x = values(T, H, DT[dtype])
    ref = R.dropout(x, p, SEED, 5)
    check(ftk().dropout_fwd(x, p, SEED, 5), ref)
    check(ftk().dropout_bwd(x, p, SEED, 5), ref)


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("H", [64, 63])
def test_strides_offsets_and_in_place(dtype, H):
    buf = values(19, 200, DT[dtype])
    for a in (0, 1, 8, 9):
        x = buf[:, a:a + H]
        ref = R.dropout(x, 0.3, SEED)
        check(ftk().dropout_fwd(x, 0.3, SEED), ref)
        out = torch.full_like(buf, 7.0)
        ftk().dropout_fwd(x, 0.3, SEED, y=out[:, 72:72 + H])
        check(out[:, 72:72 + H], ref)
        assert (out[:, :72] == 7).all() and (out[:, 72 + H:] == 7).all()
        own = buf.clone()
        assert ftk().dropout_fwd(own[:, a:a + H], 0.3, SEED, y=own[:, a:a + H]) is not None
        check(own[:, a:a + H], ref)
        own[:, a:a + H] = x
        assert torch.equal(own, buf)  # nothing beside it was touched
    one = buf[3:4, :H]  # a single row
    check(ftk().dropout_fwd(one, 0.3, SEED), R.dropout(one, 0.3, SEED))


def test_dropped_infinities_are_zero():
    x = torch.full((32, 64), float("inf"), device="cuda", dtype=torch.bfloat16)
    x[:, ::2] = float("nan")
    y = ftk().dropout_fwd(x, 0.5, 3).float().cpu()
    keep = R.keep_mask(32, 64, 0.5, 3)
    assert (y[~keep] == 0).all() and not torch.isfinite(y[keep]).any()
    assert (ftk().dropout_fwd(x, 1.0, 3) == 0).all()


@pytest.mark.parametrize("p", [2.0 ** -18, 2.0 ** -17, 1 - 2.0 ** -16, 1 - 2.0 ** -18])
def test_probabilities_at_the_ends(p):
    x = values(600, 1024, torch.bfloat16)
    check(ftk().dropout_fwd(x, p, SEED), R.dropout(x, p, SEED))


@pytest.mark.parametrize("offset, step", [(0, 0), (2 ** 32 - 1, 1), (2 ** 64 - 1, 1), (5, -3),
                                          (0x1234567890, 2 ** 40)])
def test_offset_and_step_are_one_number(offset, step):
    x = values(9, 72, torch.float32)
    s = torch.tensor([step], dtype=torch.int64, device="cuda")
    check(ftk().dropout_fwd(x, 0.4, 2 ** 64 - 1, offset, s),
          R.dropout(x, 0.4, 2 ** 64 - 1, offset, step))


def test_captured_masks_follow_the_step():
    x, step = values(40, 128, torch.bfloat16), torch.zeros(1, dtype=torch.int64, device="cuda")
    y = torch.empty_like(x)
    ftk().dropout_fwd(x, 0.2, 9, 4, step, y=y)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ftk().dropout_fwd(x, 0.2, 9, 4, step, y=y)
        dx = ftk().dropout_bwd(y, 0.2, 9, 4, step)
        step.add_(1)
    for n in range(3):
        graph.replay()
        torch.cuda.synchronize()
        check(y, R.dropout(x, 0.2, 9, 4, n))
        check(dx, R.dropout(y, 0.2, 9, 4, n))


def test_rows_past_31_bits_of_elements():
    T, H = 2 ** 19 + 3, 4104  # 2.15e9 elements
    x = torch.ones(1, device="cuda", dtype=torch.bfloat16).expand(T * H).reshape(T, H).contiguous()
    y = ftk().dropout_fwd(x, 0.5, 1)
    words = R.philox4x32((torch.arange(513).numpy()[None, :], torch.arange(T - 4, T).numpy()[:, None],
                          0, 0), (1, 0))
    import numpy as np
    half = np.stack([h for w in np.broadcast_arrays(*words)
                     for h in (w & np.uint64(0xFFFF), w >> np.uint64(16))], -1).reshape(4, -1)
    assert torch.equal(y[-4:].cpu() != 0, torch.from_numpy(half.astype(np.int64) >= 32768))
    assert abs((y[:1000] != 0).double().mean().item() - 0.5) < 2e-3


def test_another_stream_and_repeats():
    x = values(333, 896, torch.bfloat16)
    first = ftk().dropout_fwd(x, 0.1, 1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again = ftk().dropout_fwd(x, 0.1, 1)
    side.synchronize()
    assert torch.equal(first, again)


def test_autograd():
    from fine_tuning_gb300 import autograd
    x = values(33, 64, torch.float32).requires_grad_()
    step = torch.ones(1, dtype=torch.int64, device="cuda")
    g = values(33, 64, torch.float32, 1)
    autograd.dropout(x, 0.3, 7, 2, step).backward(g)
    check(x.grad, R.dropout(g, 0.3, 7, 2, 1))
    y = autograd.dropout(x, 0.3, 7, 2, step)
    step.add_(1)  # the mask of the forward pass could not be made again
    with pytest.raises(RuntimeError, match="modified"):
        y.sum().backward()
    empty = torch.empty(0, 64, device="cuda", requires_grad=True)
    autograd.dropout(empty, 0.3, 7).sum().backward()
    assert empty.grad.shape == (0, 64)
