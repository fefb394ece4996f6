"""Host-side checks of the residual stream's calls, no GPU needed: argument errors
come back as the documented status before any CUDA call (the pointers are never
dereferenced), and the binding refuses what the C calls cannot see."""
import pytest
import torch

OK, NULL, SHAPE, ALIGN, DTYPE, WORKSPACE, CUDA, ALIAS = range(8)
F32, BF16 = 0, 1
A = 1 << 20  # a fake device address, never dereferenced
M = 1 << 16
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def lib():
    from fine_tuning_gb300 import build
    build.build()
    from fine_tuning_gb300 import ftk
    return ftk.library()


def caller(f, **ok):
    def call(**kw):
        assert set(kw) <= set(ok)
        return f(*{**ok, **kw}.values())
    return call


@pytest.mark.parametrize("name", ["ftk_dropout_fwd", "ftk_dropout_bwd"])
def test_dropout_argument_errors(lib, name):
    call = caller(getattr(lib, name), x=A, ldx=64, y=A + M, ldy=64, T=4, H=64, p=0.1, seed=1,
                  offset=0, step=None, dt=BF16, s=None)
    assert call(T=0) == OK and call(T=0, x=None, y=None) == OK
    assert call(dt=2) == DTYPE
    for kw in (dict(T=-1), dict(T=1 << 31), dict(H=0), dict(H=1 << 23, ldx=1 << 23, ldy=1 << 23),
               dict(ldx=63), dict(ldy=63), dict(p=-0.1), dict(p=1.1), dict(p=NAN)):
        assert call(**kw) == SHAPE, kw
    assert call(x=None) == NULL and call(y=None) == NULL
    assert call(x=A + 1) == ALIGN and call(y=A + M + 1) == ALIGN and call(step=A + 2 * M + 4) == ALIGN
    assert call(y=A + 2) == ALIAS and call(y=A, ldy=65) == ALIAS
    assert call(step=A + M + 8) == ALIAS       # the step inside y


def test_embed_fwd_argument_errors(lib):
    call = caller(lib.ftk_embed_fwd, w=A, ldw=64, V=10, ids=A + M, x=A + 2 * M, ldx=64, T=4, H=64,
                  scale=1.0, dt=BF16, s=None)
    assert call(T=0) == OK
    assert call(dt=-1) == DTYPE
    for kw in (dict(T=-1), dict(T=1 << 31), dict(H=0), dict(V=0), dict(V=1 << 31), dict(ldw=63),
               dict(ldx=63), dict(scale=NAN), dict(scale=INF)):
        assert call(**kw) == SHAPE, kw
    for n in ("w", "ids", "x"):
        assert call(**{n: None}) == NULL
    assert call(w=A + 1) == ALIGN and call(ids=A + M + 2) == ALIGN and call(x=A + 2 * M + 1) == ALIGN
    assert call(x=A + 64) == ALIAS and call(x=A + M) == ALIAS


def test_embed_bwd_argument_errors(lib):
    ws = lib.ftk_embed_bwd_workspace_bytes(4, 64, 10)
    call = caller(lib.ftk_embed_bwd, dx=A, lddx=64, ids=A + M, dw=A + 2 * M, lddw=64, V=10, T=4,
                  H=64, scale=1.0, acc=0, ws=A + 4 * M, wsb=ws, dt=BF16, s=None)
    assert call(T=0, acc=1) == OK and call(T=0, acc=1, dx=None, ids=None, ws=None) == OK
    assert call(dt=2) == DTYPE
    for kw in (dict(T=-1), dict(T=1 << 31), dict(H=0), dict(V=0), dict(V=1 << 31), dict(lddx=63),
               dict(lddw=63), dict(scale=NAN), dict(scale=-INF)):
        assert call(**kw) == SHAPE, kw
    for n in ("dx", "ids", "dw"):
        assert call(**{n: None}) == NULL
    assert call(T=0, dw=None) == NULL          # an empty batch's gradient is all zeros
    assert call(ws=None) == WORKSPACE and call(wsb=ws - 1) == WORKSPACE
    for kw in (dict(dx=A + 1), dict(ids=A + M + 1), dict(dw=A + 2 * M + 2), dict(ws=A + 4 * M + 8)):
        assert call(**kw) == ALIGN, kw
    for kw in (dict(dw=A), dict(dw=A + M), dict(ws=A), dict(ws=A + M), dict(ws=A + 2 * M)):
        assert call(**kw) == ALIAS, kw


def test_workspace_queries(lib):
    f = lib.ftk_embed_bwd_workspace_bytes
    assert f(0, 64, 10) > 0
    assert f(-1, 64, 10) == 0 and f(4, 0, 10) == 0 and f(4, 64, 0) == 0 and f(4, 64, 1 << 31) == 0
    assert f(100000, 64, 10) >= 4 * 4 * 100000
    g = lib.ftk_rmsnorm_block_bwd_workspace_bytes
    assert g(0, 64, BF16) == 0 and g(4, 0, BF16) == 0 and g(4, 64, 5) == 0


BLOCK = dict(w_post=A + 4 * M, gate=A + 5 * M, gate_tok=A + 6 * M, w=A + 7 * M)


def test_block_fwd_argument_errors(lib):
    call = caller(lib.ftk_rmsnorm_block_fwd, x=A, ldx=64, res=A + M, ldr=64, **BLOCK, h=A + 8 * M,
                  ldh=64, y=A + 9 * M, ldy=64, r1=A + 10 * M, r=A + 11 * M, T=4, H=64, eps=1e-6,
                  res_scale=1.0, x_scale=1.0, p=0.1, seed=0, offset=0, step=A + 12 * M, dt=BF16,
                  s=None)
    assert call(T=0) == OK
    assert call(dt=9) == DTYPE
    for kw in (dict(T=-1), dict(H=0), dict(ldx=63), dict(ldr=63), dict(ldh=63), dict(ldy=63),
               dict(eps=-1e-6), dict(eps=NAN), dict(eps=INF), dict(res_scale=NAN),
               dict(x_scale=INF), dict(p=2.0)):
        assert call(**kw) == SHAPE, kw
    for n in ("x", "res", "w", "h", "y"):
        assert call(**{n: None}) == NULL, n
    for n in ("x", "res", "w_post", "gate", "w", "h", "y"):
        assert call(**{n: A + 20 * M + 1}) == ALIGN, n
    for n in ("gate_tok", "r1", "r"):
        assert call(**{n: A + 20 * M + 2}) == ALIGN, n
    assert call(step=A + 20 * M + 4) == ALIGN
    for kw in (dict(h=A + 2), dict(h=A + M + 64), dict(y=A), dict(y=A + M), dict(y=A + 8 * M),
               dict(h=A + 4 * M), dict(y=A + 7 * M), dict(r=A + 8 * M), dict(r1=A + 9 * M),
               dict(r1=A + 11 * M), dict(r=A + 6 * M), dict(step=A + 8 * M), dict(step=A + 11 * M)):
        assert call(**kw) == ALIAS, kw


def test_block_bwd_argument_errors(lib):
    call = caller(lib.ftk_rmsnorm_block_bwd, dy=A, lddy=64, dh=A + M, lddh=64, x=A + 2 * M, ldx=64,
                  h=A + 3 * M, ldh=64, **BLOCK, r1=A + 8 * M, r=A + 9 * M, dx=A + 10 * M, lddx=64,
                  dres=A + 11 * M, lddr=64, dw_post=A + 12 * M, dgate=A + 13 * M,
                  dgate_tok=A + 14 * M, dw=A + 15 * M, ws=A + 16 * M, wsb=M, T=4, H=64,
                  res_scale=1.0, x_scale=1.0, p=0.1, seed=0, offset=0, step=A + 40 * M, dt=BF16,
                  s=None)
    assert call(dt=9) == DTYPE
    for kw in (dict(T=-1), dict(H=0), dict(lddy=63), dict(lddh=63), dict(ldx=63), dict(ldh=63),
               dict(lddx=63), dict(lddr=63), dict(res_scale=INF), dict(x_scale=NAN), dict(p=NAN)):
        assert call(**kw) == SHAPE, kw
    for n in ("dy", "dh", "x", "h", "w", "r", "r1", "dx", "dres", "dw", "dw_post", "dgate",
              "dgate_tok"):
        assert call(**{n: None}) == NULL, n
    assert call(ws=None) == WORKSPACE
    for n in ("dy", "dh", "x", "h", "w_post", "gate", "w", "dx", "dres"):
        assert call(**{n: A + 50 * M + 1}) == ALIGN, n
    for n in ("gate_tok", "r1", "r", "dw", "dw_post", "dgate", "dgate_tok"):
        assert call(**{n: A + 50 * M + 2}) == ALIGN, n
    assert call(ws=A + 50 * M + 8) == ALIGN and call(step=A + 50 * M + 4) == ALIGN
    for kw in (dict(dx=A + 2), dict(dx=A + 2 * M), dict(dres=A + 3 * M), dict(dx=A, dres=A),
               dict(dres=A + 10 * M), dict(dw=A + 10 * M), dict(dw=A + 7 * M),
               dict(dgate=A + 15 * M), dict(dgate_tok=A + 6 * M), dict(dw_post=A + 13 * M),
               dict(step=A + 11 * M), dict(dw=A + 8 * M)):
        assert call(**kw) == ALIAS, kw


def test_binding_refuses(lib):
    from fine_tuning_gb300 import ftk
    x = torch.zeros(4, 8)
    ids = torch.zeros(4, dtype=torch.int32)
    for call in (lambda: ftk.dropout_fwd(x, 0.1, 1), lambda: ftk.dropout_bwd(x, 0.1, 1),
                 lambda: ftk.embed_fwd(x, ids), lambda: ftk.embed_bwd(x, ids, 4),
                 lambda: ftk.rmsnorm_block_fwd(x, x, x[0], 1e-6),
                 lambda: ftk.rmsnorm_block_bwd(x, x, x, x, x[0], x[:, 0])):
        with pytest.raises(ValueError, match="CUDA"):
            call()
    for call in (lambda: ftk.embed_fwd(x, ids.long()), lambda: ftk.embed_fwd(x, ids[::2]),
                 lambda: ftk.dropout_fwd(x.T, 0.1, 1), lambda: ftk.dropout_fwd(x[0], 0.1, 1),
                 lambda: ftk.rmsnorm_block_fwd(x, x[:2], x[0], 1e-6)):
        with pytest.raises(ValueError):
            call()
    for seed, offset in ((-1, 0), (2 ** 64, 0), (0, -1), (0, 2 ** 64)):
        with pytest.raises(ValueError, match="seed"):
            ftk._random(0.1, seed, offset, None)
    with pytest.raises(ValueError, match="step"):
        ftk._random(0.1, 0, 0, torch.zeros(2, dtype=torch.int64))
    with pytest.raises(ValueError, match="step"):
        ftk._random(0.1, 0, 0, torch.zeros(1, dtype=torch.int32))
