"""Refusals of the attention and multi-axis rotation calls, before any CUDA
call is made (the pointers below are never dereferenced), and the binding's own
checks."""
import ctypes

import numpy as np
import pytest
import torch

OK, NULL, SHAPE, ALIGN, DTYPE, WORKSPACE, CUDA, ALIAS = range(8)
F32, BF16 = 0, 1
A = 1 << 30  # a fake device address


@pytest.fixture(scope="module")
def lib():
    from fine_tuning_gb300 import build
    build.build()
    from fine_tuning_gb300 import ftk
    return ftk.library()


def caller(f, names, values):
    def call(**kw):
        a = list(values)
        for n, v in kw.items():
            a[names.index(n)] = v
        return f(*a)
    return call


STEP = 1 << 20


def fwd(lib):
    q, k, v, o, lse, cu, st = (A + i * STEP for i in range(7))
    names = ["q", "ldq", "k", "ldk", "v", "ldv", "o", "ldo", "lse", "cu", "B", "T", "Hq", "Hkv",
             "D", "scale", "causal", "status", "dt", "s"]
    return caller(lib.ftk_attn_fwd, names,
                  [q, 256, k, 128, v, 128, o, 256, lse, cu, 2, 10, 4, 2, 64, 0.125, 1, st, BF16,
                   None])


def test_attn_fwd_refusals(lib):
    call = fwd(lib)
    assert call(T=0) == OK and call(T=0, B=0) == OK
    assert call(dt=2) == DTYPE and call(dt=-1) == DTYPE
    for kw in (dict(T=-1), dict(T=1 << 31), dict(B=-1), dict(B=0), dict(Hq=0), dict(Hkv=0),
               dict(Hq=3), dict(Hq=-4), dict(Hkv=-2), dict(D=0), dict(D=257), dict(ldq=255),
               dict(ldk=127), dict(ldv=64), dict(ldo=255), dict(scale=0.0), dict(scale=-1.0),
               dict(scale=float("nan")), dict(scale=float("inf")), dict(B=(1 << 31) - 1),
               dict(T=(1 << 31) - 1, Hq=64, Hkv=2, ldq=4096, ldo=4096)):
        assert call(**kw) == SHAPE, kw
    for n in ("q", "k", "v", "o", "cu"):
        assert call(**{n: None}) == NULL, n
    for n in ("q", "k", "v", "o"):
        assert call(**{n: A + 7 * STEP + 1}) == ALIGN, n
    for n in ("lse", "cu", "status"):
        assert call(**{n: A + 7 * STEP + 2}) == ALIGN, n
    for n in ("q", "k", "v", "cu", "status"):
        assert call(**{n: A + 3 * STEP + 64}) == ALIAS, n  # inside o
        assert call(**{n: A + 4 * STEP + 64}) == ALIAS, n  # inside lse
    assert call(lse=A + 3 * STEP + 256) == ALIAS
    # slices of one fused buffer are apart; a slice one element off is not
    fused = dict(q=A, ldq=512, k=A + 512, ldk=512, v=A + 768, ldv=512)
    assert call(T=0, **fused) == OK
    assert call(o=A + 2, ldo=512, **fused) == ALIAS


def bwd(lib):
    ptr = {n: A + i * STEP for i, n in enumerate(
        ["do", "q", "k", "v", "o", "lse", "dq", "dk", "dv", "ws", "cu", "status"])}
    names, values = [], []
    for n, ld in (("do", 256), ("q", 256), ("k", 128), ("v", 128), ("o", 256)):
        names += [n, "ld" + n]
        values += [ptr[n], ld]
    names += ["lse"]
    values += [ptr["lse"]]
    for n, ld in (("dq", 256), ("dk", 128), ("dv", 128)):
        names += [n, "ld" + n]
        values += [ptr[n], ld]
    names += ["ws", "wsb", "cu", "B", "T", "Hq", "Hkv", "D", "scale", "causal", "status", "dt", "s"]
    values += [ptr["ws"], 1 << 16, ptr["cu"], 2, 10, 4, 2, 64, 0.125, 1, ptr["status"], BF16, None]
    return caller(lib.ftk_attn_bwd, names, values), ptr


def test_attn_bwd_refusals(lib):
    call, ptr = bwd(lib)
    assert call(T=0) == OK
    assert call(dt=5) == DTYPE
    for kw in (dict(T=-1), dict(B=0), dict(Hq=3), dict(D=0), dict(D=300), dict(lddo=255),
               dict(ldq=0), dict(ldk=127), dict(ldv=127), dict(ldo=1), dict(lddq=255),
               dict(lddk=127), dict(lddv=127), dict(scale=0.0)):
        assert call(**kw) == SHAPE, kw
    for n in ("do", "q", "k", "v", "o", "lse", "dq", "dk", "dv", "cu"):
        assert call(**{n: None}) == NULL, n
    assert call(ws=None) == WORKSPACE
    need = lib.ftk_attn_bwd_workspace_bytes(10, 4, 2, 64, BF16)
    assert need >= 10 * 4 * 4
    assert call(wsb=need - 1) == WORKSPACE
    for n in ("do", "q", "k", "v", "o", "dq", "dk", "dv"):
        assert call(**{n: A + 13 * STEP + 1}) == ALIGN, n
    assert call(ws=A + 13 * STEP + 8) == ALIGN and call(lse=A + 13 * STEP + 2) == ALIGN
    for out in ("dq", "dk", "dv", "ws"):
        for n in ("do", "q", "k", "v", "o", "lse", "cu", "status"):
            assert call(**{n: ptr[out] + 64}) == ALIAS, (out, n)
    assert call(dk=ptr["dq"]) == ALIAS and call(dv=ptr["dk"]) == ALIAS
    assert call(ws=ptr["dv"] + 128) == ALIAS


def test_attn_workspace_of_nothing(lib):
    f = lib.ftk_attn_bwd_workspace_bytes
    assert f(0, 4, 2, 64, BF16) == 0 and f(-5, 4, 2, 64, BF16) == 0
    assert f(10, 3, 2, 64, BF16) == 0 and f(10, 4, 2, 0, BF16) == 0 and f(10, 4, 2, 64, 9) == 0


@pytest.mark.parametrize("name", ["ftk_qk_mrope_fwd", "ftk_qk_mrope_bwd"])
def test_mrope_refusals(lib, name):
    q, k, qo, ko, pos = (A + i * STEP for i in range(5))
    axis = (ctypes.c_int32 * 8)(0, 0, 1, 1, 1, 2, 2, 2)
    freq = (ctypes.c_double * 8)(*[2.0 ** -i for i in range(8)])
    names = ["q", "ldq", "k", "ldk", "qo", "ldqo", "ko", "ldko", "pos", "ldp", "axes", "axis", "T",
             "Hq", "Hkv", "D", "theta", "freq", "dt", "s"]
    call = caller(getattr(lib, name), names,
                  [q, 64, k, 32, qo, 64, ko, 32, pos, 10, 3, ctypes.addressof(axis), 10, 4, 2, 16,
                   1e4, None, BF16, None])
    assert call(T=0) == OK
    assert call(dt=3) == DTYPE
    for kw in (dict(T=-1), dict(ldp=9), dict(axes=0), dict(axes=2), dict(axes=257), dict(D=15),
               dict(D=0), dict(D=514), dict(Hq=0, Hkv=0), dict(Hq=-1), dict(Hkv=-1), dict(ldq=63),
               dict(ldko=31), dict(theta=0.0), dict(theta=float("nan"))):
        assert call(**kw) == SHAPE, kw
    bad = (ctypes.c_int32 * 8)(0, 0, 1, -1, 1, 2, 2, 2)
    assert call(axis=ctypes.addressof(bad)) == SHAPE
    for x in (1.5, -0.5, float("nan")):
        freq[3] = x
        assert call(freq=ctypes.addressof(freq)) == SHAPE, x
    for n in ("q", "k", "qo", "ko", "pos", "axis"):
        assert call(**{n: None}) == NULL, n
    assert call(q=q + 1) == ALIGN and call(ko=ko + 1) == ALIGN and call(pos=pos + 2) == ALIGN
    assert call(qo=q + 2) == ALIAS and call(qo=q, ldqo=72) == ALIAS  # over q, but not q itself
    assert call(qo=k) == ALIAS and call(ko=qo + 64) == ALIAS and call(pos=qo + 64) == ALIAS


def test_binding_checks():
    from fine_tuning_gb300 import ftk
    assert ftk.mrope_axis_of((1, 0, 3)).tolist() == [0, 2, 2, 2]
    for bad in ((), (-1, 2), (0, 0), (1.5, 2)):
        with pytest.raises(ValueError):
            ftk.mrope_axis_of(bad)
    x = torch.zeros(4, 2, 8)
    with pytest.raises(ValueError):  # not on a GPU
        ftk.attn_fwd(x, x, x, torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError):
        ftk.qk_mrope_fwd(x, x, torch.zeros(3, 4, dtype=torch.int32), np.zeros(4, np.int32), 1e4)
    with pytest.raises(ValueError):
        ftk.qk_mrope_fwd(None, None, torch.zeros(3, 4, dtype=torch.int32), np.zeros(4), 1e4)


def test_attn_workspace_does_not_grow_with_the_group(lib):
    """The fp32 sums of dk and dv that the workspace holds beside delta: at most
    two shares more than 304 tasks over the key tiles' sums give."""
    f = lib.ftk_attn_bwd_workspace_bytes
    for T, Hkv, G, D in ((38784, 1, 64, 128), (38784, 1, 128, 128), (38912, 1, 128, 64),
                         (19400, 2, 32, 64), (8192, 1, 8, 128), (2048, 8, 4, 128),
                         (16384, 2, 7, 64), (100, 1, 256, 8), (1, 1, 1, 8)):
        sums = -(-T // 128) * Hkv
        delta = -(-T * Hkv * G * 4 // 16) * 16
        shares, rest = divmod(f(T, Hkv * G, Hkv, D, BF16) - delta, 2 * T * Hkv * D * 4)
        assert rest == 0 and shares != 1
        assert shares <= min(G, 304 // sums + 2), (T, Hkv, G, D)


def test_status_bits_of_the_header_and_the_kernels_agree():
    import os
    import re
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    header = open(os.path.join(root, "include", "ftk.h")).read()
    csrc = os.path.join(root, "fine_tuning_gb300", "csrc")
    kernels = "".join(open(os.path.join(csrc, f)).read() for f in ("common.cuh", "attn_tc.cuh"))
    for a, b in (("WAIT_TIMEOUT", "WaitTimeout"), ("SMEM_BASE", "SmemBase")):
        x = re.search(rf"#define FTK_DEVSTAT_{a} (\d)u", header).group(1)
        assert x == re.search(rf"kStatus{b} = (\d)u", kernels).group(1)
    # the one kernel that cannot align its tiles by hand looks before it uses them
    bwd = open(os.path.join(root, "fine_tuning_gb300", "csrc", "attn_bwd_tc.cu")).read()
    at = bwd.index("__align__(1024) unsigned char smem_aligned[]")
    look, wait = bwd.index("kStatusSmemBase", at), bwd.index("pdl_wait();", at)
    assert look < wait < bwd.index("return;", at) < bwd.index("mbar_init", at)


def test_attn_refuses_rows_that_32_bits_do_not_count(lib):
    """The last tile's rows reach up to 127 past the last token."""
    big = dict(Hq=1, Hkv=1, D=8, B=1, ldq=8, ldk=8, ldv=8, ldo=8)
    call, (back, _) = fwd(lib), bwd(lib)
    for T in ((1 << 31) - 1, (1 << 31) - 128, (1 << 31) - 1023):
        assert call(T=T, **big) == SHAPE, T
        assert back(T=T, lddo=8, lddq=8, lddk=8, lddv=8, **big) == SHAPE, T
        assert lib.ftk_attn_bwd_workspace_bytes(T, 1, 1, 8, BF16) == 0
    # refused for the overlap of the pointers below, so not for the size
    assert call(T=(1 << 31) - 1024, **big) == ALIAS


def test_attn_refuses_scales_whose_exponent_base_two_overflows(lib):
    """The exponentials are powers of two, of scores times scale * log2(e)."""
    call, (back, _) = fwd(lib), bwd(lib)
    for scale in (2.5e38, 3.4e38):
        assert call(scale=scale) == SHAPE and back(scale=scale) == SHAPE
    assert call(scale=2.0 ** 127, o=A) == ALIAS  # refused for the overlap alone


def test_attention_is_no_part_of_the_sources_that_measured_traffic_is_filed_under():
    """The DRAM traffic on file counts while an op's sources and the shared headers are
    those of its capture; what only attention needs must not touch them."""
    import os
    import bench
    csrc = os.path.join(bench.ROOT, "fine_tuning_gb300", "csrc")
    names = {n for names in bench.KERNEL_SOURCES.values() for n in names}
    for name in sorted(names | {"common.cuh", "launch.h"}):
        text = open(os.path.join(csrc, name)).read()
        for word in ("Attn", "attn_", "Mrope", "mrope"):
            assert word not in text, f"{name}: {word}"
