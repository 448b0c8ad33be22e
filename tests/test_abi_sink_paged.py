"""Refusals of the SW-SKA entry points with first tokens that stay visible and of the paged cache's: every bad argument is
answered on the host with its status before anything is launched (no call below reaches a kernel)."""
import ctypes

import pytest
import torch

import sliding_window_attention_chunked_b200 as rod
from sliding_window_attention_chunked_b200 import build as rbuild

OK, NULL, SHAPE, ALIGN, DTYPE, WS = 0, -1, -2, -3, -4, -5
P, MIS, MIS2 = ctypes.c_void_p(0x10000), ctypes.c_void_p(0x10008), ctypes.c_void_p(0x10002)
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def lib():
    rbuild.build()
    return rod.load_library()


def caller(fn, **base):
    return lambda **kw: fn(*{**base, **kw}.values())


def test_sink_prefill(lib):
    f = caller(lib.rod_swska_sink_prefill, q=P, k=P, v=P, o=P, lse=P, B=1, H=2, T=8, dk=16, dv=32, W=4, S=2, scale=0.0, dt=2, s=None)
    assert f(dt=3) == DTYPE
    for bad in (dict(W=0), dict(S=-1), dict(S=129), dict(dk=24), dict(dv=256), dict(H=65), dict(T=-1), dict(B=-1), dict(scale=NAN), dict(scale=INF)):
        assert f(**bad) == SHAPE, bad
    for n in ("q", "k", "v", "o", "lse"):
        assert f(**{n: None}) == NULL
    for n in ("q", "k", "v", "o"):
        assert f(**{n: MIS}) == ALIGN
    assert f(lse=MIS2) == ALIGN
    assert f(T=0, q=None) == OK and f(B=0, q=None) == OK and f(H=0, q=None) == OK


def test_sink_backward(lib):
    need = lib.rod_swska_sink_backward_workspace_size(1, 2, 8, 16, 32, 4, 2)
    assert need > 0
    f = caller(lib.rod_swska_sink_backward, q=P, k=P, v=P, o=P, lse=P, dO=P, dq=P, dk=P, dv=P, B=1, H=2, T=8, dkd=16, dvd=32, W=4, S=2,
               scale=0.0, dt=2, ws=P, wsb=need, s=None)
    assert f(dt=0) == DTYPE
    for bad in (dict(W=0), dict(S=-1), dict(S=129), dict(dkd=8), dict(dvd=0), dict(H=65), dict(T=-1), dict(scale=NAN)):
        assert f(**bad) == SHAPE, bad
    for n in ("q", "k", "v", "o", "lse", "dO", "dq", "dk", "dv"):
        assert f(**{n: None}) == NULL
    for n in ("q", "k", "v", "o", "dO", "dq", "dk", "dv"):
        assert f(**{n: MIS}) == ALIGN
    assert f(lse=MIS2) == ALIGN
    assert f(ws=None) == WS and f(wsb=need - 1) == WS and f(ws=MIS) == ALIGN
    assert f(T=0, q=None) == OK
    assert lib.rod_swska_sink_backward_workspace_size(1, 2, 8, 24, 32, 4, 2) == 0
    # more far segments need more room, and a window as long as the sequence needs none
    size = lambda W, S: lib.rod_swska_sink_backward_workspace_size(1, 2, 4096, 128, 128, W, S)
    assert size(128, 4) > size(4096, 4) == size(4096, 0) == size(10 ** 9, 128)


def test_extend_paged(lib):
    need = lib.rod_swska_extend_paged_workspace_size(10, 3, 2, 128, 128, 4, 1)
    assert need > 0
    f = caller(lib.rod_swska_extend_paged, q=P, kn=P, vn=P, kp=P, vp=P, t=P, sl=P, cu=P, ctx=P, o=P, M=10, N=3, H=2, dk=128, dv=128, P=20,
               page=16, mp=4, W=8, S=4, ml=4, scale=0.0, dt=1, ws=P, wsb=need, s=None)
    assert f(dt=7) == DTYPE
    for bad in (dict(page=12), dict(page=0), dict(page=4), dict(mp=0), dict(P=0), dict(W=0), dict(S=-1), dict(S=129), dict(H=0), dict(H=65),
                dict(dk=96), dict(M=-1), dict(N=-1), dict(N=16385), dict(ml=-1), dict(P=2 ** 30), dict(mp=2 ** 28), dict(scale=NAN)):
        assert f(**bad) == SHAPE, bad
    for n in ("q", "kp", "vp", "t", "cu", "ctx", "o", "kn", "vn", "sl"):
        assert f(**{n: None}) == NULL, n
    for n in ("q", "kn", "vn", "kp", "vp", "o"):
        assert f(**{n: MIS}) == ALIGN
    for n in ("t", "sl", "cu", "ctx"):
        assert f(**{n: MIS2}) == ALIGN
    assert f(ws=None) == WS and f(wsb=need - 1) == WS and f(ws=MIS) == ALIGN
    assert f(M=0, q=None) == OK and f(N=0, q=None) == OK


def test_page_tables(lib):
    f = caller(lib.rod_swska_page_tables, ctx=P, new=P, t=P, first=P, fl=P, fc=P, cu=P, slot=P, N=3, mp=4, P=20, page=16, W=8, S=4, M=10, s=None)
    for bad in (dict(N=-1), dict(N=16385), dict(mp=0), dict(P=0), dict(page=0), dict(W=0), dict(S=-1), dict(M=-1), dict(P=2 ** 30), dict(mp=2 ** 28)):
        assert f(**bad) == SHAPE, bad
    for n in ("ctx", "new", "t", "first", "fl", "fc", "cu", "slot"):
        assert f(**{n: None}) == NULL, n
    for n in ("ctx", "new", "t", "first", "fl", "fc", "cu"):
        assert f(**{n: MIS2}) == ALIGN
    assert f(slot=MIS) == ALIGN


def test_binding_refuses_cpu_tensors_and_mixed_arguments():
    z = torch.zeros
    with pytest.raises(ValueError, match="CUDA"):
        rod.swska_sink_prefill(z(1, 2, 8, 16), z(1, 8, 16), z(1, 2, 8, 32), 4, 2)
    with pytest.raises(ValueError, match="CUDA"):
        rod.swska_sink_backward(*(z(1, 2, 8, 16), z(1, 8, 16), z(1, 2, 8, 32)), z(1, 2, 8, 32), z(1, 2, 8), z(1, 2, 8, 32), 4, 2)
    with pytest.raises(ValueError, match="CUDA"):
        rod.swska_extend_paged(z(1, 2, 16), None, None, z(1, 8, 16), z(1, 2, 8, 16), z(1, 1, dtype=torch.int32), None,
                               z(2, dtype=torch.int32), z(1, dtype=torch.int64), 4)
    with pytest.raises(ValueError, match="CUDA"):
        i = z(1, dtype=torch.int32)
        rod.swska_page_tables(z(1, dtype=torch.int64), i, z(1, 1, dtype=torch.int32), i, i, i, 8, 4, 0, 1)
