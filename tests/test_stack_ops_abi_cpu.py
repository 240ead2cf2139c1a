"""Host-side checks of the dense recurrence, residual norm and balance entry
points (no GPU): invalid arguments are refused before any launch."""
import ctypes
import os

import pytest

from sparse_memory_linear_amd import binding

P = ctypes.c_void_p
FAKE = P(4096)  # never dereferenced: every call below fails its checks or is empty work
F = ctypes.c_float


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(binding.LIB_PATH):
        import __graft_entry__
        __graft_entry__.build()
    return binding.lib()


def test_dense_scan_checks(lib):
    base = dict(q=FAKE, k=FAKE, v=FAKE, dt=1, a=FAKE, b=FAKE, S0=FAKE, S=FAKE, y=FAKE, B=2, H=2, T=4096, dk=64, dv=64,
                ws=FAKE, wsb=1 << 40, st=None)
    call = lambda **kw: lib.sdm_dense_scan_forward(*dict(base, **kw).values())  # noqa: E731
    for n in ("q", "k", "v", "a", "b", "y"):
        assert call(**{n: None}) == 1, n
        assert call(**{n: P(4104)}) == 4, n
    assert call(S0=P(4100)) == 4 and call(S=P(4100)) == 4
    assert call(dt=2) == 3 and call(dt=-1) == 3
    assert call(T=-1) == 2 and call(dk=0) == 2
    assert call(dk=12) == 5 and call(dv=264) == 5
    assert call(B=1 << 31) == 5 and call(B=1 << 20, H=1 << 10, T=1 << 20) == 5 and call(T=1 << 62) == 5
    assert call(ws=None) == 7 and call(wsb=16) == 7 and call(ws=P(4100)) == 4
    assert call(B=0, q=None, k=None, v=None, a=None, b=None, y=None, S0=None, S=None) == 0
    assert call(T=0, q=None, k=None, v=None, a=None, b=None, y=None) == 0  # S is S0: nothing to pass on
    assert lib.sdm_dense_scan_workspace_bytes(2, 2, 8, 64, 64) == 0
    assert lib.sdm_dense_scan_workspace_bytes(2, 2, 0, 64, 64) == 0
    assert lib.sdm_dense_scan_workspace_bytes(2, 2, 100, 63, 64) == -1
    assert lib.sdm_dense_scan_workspace_bytes(-1, 2, 100, 64, 64) == -1


def test_dense_scan_backward_checks(lib):
    base = dict(q=FAKE, k=FAKE, v=FAKE, dt=1, a=FAKE, b=FAKE, dy=FAKE, S0=FAKE, dS=FAKE, dq=FAKE, dk=FAKE, dv=FAKE,
                dla=FAKE, db=FAKE, dS0=FAKE, B=2, H=2, T=100, dks=64, dvs=64, ws=FAKE, wsb=1 << 40, st=None)
    call = lambda **kw: lib.sdm_dense_scan_backward(*dict(base, **kw).values())  # noqa: E731
    for n in ("q", "k", "v", "a", "b", "dy", "dq", "dk", "dv", "dla", "db"):
        assert call(**{n: None}) == 1, n
    for n in ("dy", "S0", "dS", "dS0"):
        assert call(**{n: P(4104)}) == 4, n
    assert call(dt=7) == 3 and call(H=-1) == 2 and call(dks=260) == 5
    assert call(ws=None) == 7 and call(wsb=1) == 7
    assert call(H=0, q=None, dy=None) == 0
    assert lib.sdm_dense_scan_backward_workspace_bytes(0, 2, 100, 64, 64) == 0
    assert lib.sdm_dense_scan_backward_workspace_bytes(2, 2, 100, 64, 512) == -1


@pytest.mark.parametrize("B,H,T,dk,dv", [(1 << 21, 1, 1, 8, 8), (64, 1 << 14, 512, 8, 72), (1 << 20, 1, 1, 128, 128),
                                         (1 << 14, 16, 0, 256, 256), (512, 2, 1 << 20, 8, 8)])
def test_dense_sizes_beyond_a_launch_are_refused(lib, B, H, T, dk, dv):
    assert lib.sdm_dense_scan_forward(*[FAKE] * 3, 1, *[FAKE] * 5, B, H, T, dk, dv, FAKE, 1 << 60, None) == 5
    assert lib.sdm_dense_scan_backward(*[FAKE] * 3, 1, *[FAKE] * 11, B, H, T, dk, dv, FAKE, 1 << 60, None) == 5


def test_residual_norm_checks(lib):
    x, r, h, y = P(4096), P(8192), P(12288), P(16384)
    base = dict(x=x, xd=1, r=r, h=h, hd=1, g=FAKE, eps=F(1e-6), rows=4, d=256, y=y, yd=2, s=FAKE, grp=128, st=None)
    call = lambda **kw: lib.sdm_residual_norm(*dict(base, **kw).values())  # noqa: E731
    assert call(xd=2) == 3 and call(hd=2) == 3 and call(yd=3) == 3
    assert call(rows=-1) == 2 and call(d=0) == 2 and call(eps=F(-1.0)) == 2 and call(eps=F(float("nan"))) == 2
    assert call(d=16640) == 5 and call(rows=1 << 31) == 5
    assert call(grp=96) == 5 and call(grp=16) == 5 and call(grp=1024, d=2048) == 5 and call(grp=128, d=192) == 5
    assert call(yd=1) == 2                                   # groups need an e4m3 output
    for n in ("x", "g", "y", "s"):
        assert call(**{n: None}) == 1, n
        assert call(**{n: P(4100)}) == 4, n
    assert call(r=None) == 1 and call(h=None) == 1          # both or neither
    assert call(y=x) == 2 and call(y=h) == 2 and call(y=r) == 2
    assert call(h=x, xd=0) == 2
    assert call(rows=0, x=None, r=None, h=None, g=None, y=None, s=None) == 0
    bwd = dict(dy=x, dh=r, gd=1, h=h, hd=1, g=FAKE, eps=F(1e-6), rows=4, d=256, dx=y, dg=FAKE, ws=FAKE, wsb=1 << 30, st=None)
    callb = lambda **kw: lib.sdm_residual_norm_backward(*dict(bwd, **kw).values())  # noqa: E731
    for n in ("dy", "h", "g", "dx", "dg"):
        assert callb(**{n: None}) == 1, n
    assert callb(gd=2) == 3 and callb(hd=9) == 3 and callb(dh=P(4100)) == 4 and callb(dx=h, hd=0) == 2
    assert callb(ws=None) == 7 and callb(wsb=8) == 7
    assert callb(rows=0, dy=None, h=None, dx=None, dg=None) == 0
    assert lib.sdm_residual_norm_backward_workspace_bytes(0, 64) == 0
    assert lib.sdm_residual_norm_backward_workspace_bytes(5, 0) == -1
    assert lib.sdm_residual_norm_backward_workspace_bytes(5, 16385) == -1


def test_balance_checks(lib):
    base = dict(i=FAKE, w=FAKE, m=None, B=2, H=2, T=16, K=8, N=256, c=FAKE, ms=FAKE, t=FAKE, lo=FAKE, ws=FAKE,
                wsb=1 << 30, st=None)
    call = lambda **kw: lib.sdm_balance_forward(*dict(base, **kw).values())  # noqa: E731
    for n in ("i", "w", "c", "ms", "t", "lo"):
        assert call(**{n: None}) == 1, n
        assert call(**{n: P(4100)}) == 4, n
    assert call(T=-1) == 2 and call(K=0) == 2 and call(N=0) == 2
    assert call(N=(1 << 18) + 1) == 5 and call(K=257) == 5 and call(H=4097) == 5
    assert call(B=1 << 16, T=1 << 12) == 5                   # 2^31 selections a head
    assert call(B=1 << 62, T=1 << 62) == 5
    assert call(ws=None) == 7 and call(wsb=100) == 7
    assert call(H=0, i=None, w=None, c=None, ms=None, t=None, lo=None) == 0
    bwd = dict(i=FAKE, m=None, c=FAKE, t=FAKE, dl=FAKE, B=2, H=2, T=16, K=8, N=256, d=FAKE, st=None)
    callb = lambda **kw: lib.sdm_balance_backward(*dict(bwd, **kw).values())  # noqa: E731
    for n in ("i", "c", "t", "dl", "d"):
        assert callb(**{n: None}) == 1, n
    assert callb(K=300) == 5 and callb(N=-1) == 2
    assert callb(T=0, i=None, c=None, t=None, dl=None, d=None) == 0
    assert lib.sdm_balance_workspace_bytes(1, 1, 1, 0, 4) == -1


def test_binding_refuses_cpu_tensors(lib):
    import torch
    q, g = torch.zeros(1, 1, 4, 8), torch.zeros(1, 1, 4)
    i, w = torch.zeros(1, 1, 4, 2, dtype=torch.int32), torch.zeros(1, 1, 4, 2)
    for call in (lambda: binding.sdm_dense_scan_forward(q, q, q, g, g),
                 lambda: binding.sdm_dense_scan_backward(q, q, q, g, g, q),
                 lambda: binding.sdm_residual_norm(q, torch.ones(8)),
                 lambda: binding.sdm_residual_norm_backward(q, q, torch.ones(8)),
                 lambda: binding.sdm_balance_forward(i, w, 4)):
        with pytest.raises(ValueError):
            call()


@pytest.mark.parametrize("B,H,T,dk,dv", [(1 << 21, 1, 1, 8, 8), (64, 1 << 14, 512, 8, 72), (1 << 20, 1, 1, 128, 128),
                                         (512, 2, 1 << 20, 8, 8), ((1 << 31) - 1, 1, (1 << 31) - 1, 256, 256),
                                         (1 << 29, 1, 1 << 24, 256, 256), (32768, 65534, (1 << 31) - 1, 256, 256)])
def test_refused_dense_sizes_have_no_workspace(lib, B, H, T, dk, dv):
    assert lib.sdm_dense_scan_workspace_bytes(B, H, T, dk, dv) == -1
    assert lib.sdm_dense_scan_backward_workspace_bytes(B, H, T, dk, dv) == -1
    for f in (binding.sdm_dense_scan_workspace_bytes, binding.sdm_dense_scan_backward_workspace_bytes):
        with pytest.raises(ValueError):
            f(B, H, T, dk, dv)
