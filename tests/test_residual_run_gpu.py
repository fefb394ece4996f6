"""The residual stream's operators as a step uses them: lookup, two blocks that join
the stream, the tied head's loss, and back to the table's gradient; eager against a
composition in 64 bits, captured, from several threads."""
import threading

import pytest
import torch

from oracle import residual as R

pytestmark = pytest.mark.gpu
T, H, V, I, EPS, P, SEED = 96, 128, 300, 256, 1e-6, 0.1, 42


def weights(dtype):
    g = torch.Generator(device="cuda").manual_seed(0)
    rand = lambda std, *s: (std * torch.randn(*s, generator=g, device="cuda")).to(dtype)
    one = lambda: (1 + 0.1 * torch.randn(H, generator=g, device="cuda")).to(dtype)
    return {"W": rand(0.5, V, H), "n0": one(), **{f"up{i}": rand(H ** -0.5, 2 * I, H) for i in (0, 1)},
            **{f"down{i}": rand(I ** -0.5, H, I) for i in (0, 1)},
            **{f"{n}{i}": one() for n in ("post", "pre") for i in (0, 1)},
            **{f"gate{i}": one() for i in (0, 1)}}


def batch():
    g = torch.Generator(device="cuda").manual_seed(1)
    ids = torch.randint(0, V, (T,), generator=g, device="cuda", dtype=torch.int32)
    ids[-7:] = -100
    y = torch.cat([ids[1:], ids[-1:]])
    return ids, y


def step_of(w, ids, y, step):
    """One forward pass through the library's autograd operators."""
    from fine_tuning_gb300 import autograd as ag
    s = ag.embedding(w["W"], ids, H ** 0.5 / 8)
    s = ag.dropout(s, P, SEED, 0, step)
    n = ag.rmsnorm(s, w["n0"], EPS)
    for i in (0, 1):
        gu = n @ w[f"up{i}"].T
        b = ag.swiglu(gu[:, :I], gu[:, I:]) @ w[f"down{i}"].T
        s, n = ag.rmsnorm_block(b, s, w[f"pre{i}"], EPS, w[f"post{i}"], w[f"gate{i}"], None, 1.0, 0.7,
                                P, SEED, 1 + i, step)
    return n, ag.cross_entropy_head(n, w["W"], y) if n.dtype == torch.bfloat16 else \
        head64(n.float(), w["W"].float(), y)


def head64(n, W, y):
    ok = (y >= 0) & (y < V)
    z = n @ W.T
    pick = z.gather(1, y.clamp(0).long()[:, None])[:, 0]
    return ((z.logsumexp(1) - pick) * ok).sum() / ok.sum()


def plain(w, ids, y, step):
    """The same in 64 bits, from torch's elementary operations."""
    def drop(x, offset):
        return torch.where(R.keep_mask(T, H, P, SEED, offset, step).cuda(), x * R.drop_scale(P), 0.0)

    def norm(x, weight):
        return x * (x.square().mean(1, keepdim=True) + EPS) ** -0.5 * weight

    there = (ids >= 0) & (ids < V)
    s = torch.where(there[:, None], w["W"][ids.clamp(0).long()] * (H ** 0.5 / 8), 0.0)
    s = drop(s, 0)
    n = norm(s, w["n0"])
    for i in (0, 1):
        gu = n @ w[f"up{i}"].T
        b = torch.nn.functional.silu(gu[:, :I]) * gu[:, I:] @ w[f"down{i}"].T
        s = s + 0.7 * drop(norm(b, w[f"post{i}"]) * w[f"gate{i}"], 1 + i)
        n = norm(s, w[f"pre{i}"])
    return n, head64(n, w["W"], y)


def grads_of(w, forward):
    leaf = {k: v.detach().requires_grad_() for k, v in w.items()}
    n, loss = forward(leaf)
    return n.detach(), loss.detach(), dict(zip(leaf, torch.autograd.grad(loss, list(leaf.values()))))


def test_step_against_64_bits():
    w, (ids, y) = weights(torch.float32), batch()
    step = torch.tensor([3], device="cuda")
    n, loss, g = grads_of(w, lambda v: step_of(v, ids, y, step))
    n64, loss64, g64 = grads_of({k: v.double() for k, v in w.items()}, lambda v: plain(v, ids, y, 3))
    # five layers of fp32 operations with sums of up to 256 terms: each is off by at most some
    # 256 u of its terms' size, and the norms keep those near 1; 2^-12 leaves a factor of 4
    close = lambda a, b: (a.double() - b).abs().max() <= 2.0 ** -12 * b.abs().max()
    assert close(n, n64) and close(loss, loss64)
    for k in g:
        assert close(g[k], g64[k]), k


def test_captured_step_follows_its_eager_one():
    w, (ids, y) = weights(torch.bfloat16), batch()
    leaf = {k: v.detach().requires_grad_() for k, v in w.items()}
    step = torch.zeros(1, dtype=torch.int64, device="cuda")

    def go():
        n, loss = step_of(leaf, ids, y, step)
        return (n, loss, *torch.autograd.grad(loss, list(leaf.values())))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(2):
            go()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = go()
        step.add_(1)
    for i in range(3):
        step.fill_(10 + i)
        graph.replay()
        torch.cuda.synchronize()
        kept = [t.clone() for t in out]
        step.fill_(10 + i)
        for a, b in zip(kept, go()):
            assert torch.equal(a, b)
    from fine_tuning_gb300 import ftk
    assert ftk.device_status() == 0


def test_steps_from_several_threads():
    w, (ids, y) = weights(torch.bfloat16), batch()
    step = torch.zeros(1, dtype=torch.int64, device="cuda")
    _, loss, g = grads_of(w, lambda v: step_of(v, ids, y, step))
    torch.cuda.synchronize()
    bad = []

    def work():
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(4):
                    _, l2, g2 = grads_of(w, lambda v: step_of(v, ids, y, step))
                    torch.cuda.current_stream().synchronize()
                    if not (torch.equal(loss, l2) and all(torch.equal(g[k], g2[k]) for k in g)):
                        bad.append("differs")
        except Exception as e:  # noqa: BLE001
            bad.append(repr(e))

    threads = [threading.Thread(target=work) for _ in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad
