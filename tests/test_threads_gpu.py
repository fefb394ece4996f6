"""Calls whose thread has made no CUDA call before (a data loader's, a server's or
autograd's worker): all buffers exist, so the library's call is the first."""
import threading

import pytest
import torch

from fine_tuning_gb300 import build, ftk

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    ftk.library()
    yield
    assert ftk.device_status(clear=True) == 0


def first_in_a_thread(call):
    torch.cuda.synchronize()
    failed = []

    def work():
        try:
            call()
        except Exception as e:  # noqa: BLE001
            failed.append(e)

    t = threading.Thread(target=work)
    t.start()
    t.join()
    if failed:
        raise failed[0]
    torch.cuda.synchronize()


def rnd(*shape, seed=0):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return torch.randn(shape, generator=g, device=DEV).bfloat16()


def test_cross_entropy():
    h, W = rnd(300, 64), rnd(1000, 64, seed=1)
    y = torch.arange(300, dtype=torch.int32, device=DEV)
    loss, lse = ftk.cce_fwd(h, W, y)
    one = torch.ones(1, device=DEV)
    dh, dW = ftk.cce_bwd(h, W, y, lse, one)
    ws = torch.empty(1 << 24, dtype=torch.uint8, device=DEV)
    out = [torch.zeros_like(t) for t in (loss, lse, dh, dW)]
    first_in_a_thread(lambda: ftk.cce_fwd(h, W, y, loss=out[0], lse=out[1], workspace=ws))
    first_in_a_thread(lambda: ftk.cce_bwd(h, W, y, lse, one, dh=out[2], dW=out[3], workspace=ws))
    for a, b in zip(out, (loss, lse, dh, dW)):
        assert torch.equal(a, b)


def test_gemm():
    a, b = rnd(200, 64), rnd(256, 64, seed=1)
    ref, c = ftk.gemm_bf16(a, b), torch.zeros(200, 256, device=DEV)
    first_in_a_thread(lambda: ftk.gemm_bf16(a, b, c=c))
    assert torch.equal(ref, c)


@pytest.mark.parametrize("D", [64, 128])
def test_attention(D):
    q, k, v, do = (rnd(200, h, D, seed=i) for i, h in enumerate((4, 2, 2, 4)))
    cu = torch.tensor([0, 77, 200], dtype=torch.int32, device=DEV)
    o, lse = ftk.attn_fwd(q, k, v, cu)
    ref = ftk.attn_bwd(do, q, k, v, o, lse, cu)
    o2, lse2 = torch.zeros_like(o), torch.zeros_like(lse)
    out = [torch.zeros_like(t) for t in ref]
    ws = torch.empty(ftk.attn_bwd_workspace_bytes(200, 4, 2, D, q.dtype), dtype=torch.uint8,
                     device=DEV)
    first_in_a_thread(lambda: ftk.attn_fwd(q, k, v, cu, o=o2, lse=lse2))
    first_in_a_thread(lambda: ftk.attn_bwd(do, q, k, v, o, lse, cu, dq=out[0], dk=out[1],
                                           dv=out[2], workspace=ws))
    for a, b in zip((o2, lse2, *out), (o, lse, *ref)):
        assert torch.equal(a, b)


def test_several_threads_at_once():
    xs = [(rnd(200 + 64 * i, 64, seed=i), rnd(256, 64, seed=9)) for i in range(4)]
    ref = [ftk.gemm_bf16(a, b) for a, b in xs]
    got = [None] * len(xs)

    def work(i):
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(10):
                got[i] = ftk.gemm_bf16(*xs[i])
            torch.cuda.current_stream().synchronize()

    torch.cuda.synchronize()
    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(xs))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    for a, b in zip(got, ref):
        assert torch.equal(a, b)
