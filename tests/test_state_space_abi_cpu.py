"""Host-side checks of the causal convolution, the selective scan and the layer norm (no GPU):
invalid arguments are refused before any launch."""
import ctypes
import os

import pytest

from sparse_memory_linear_amd import binding

P = ctypes.c_void_p
FAKE = P(4096)  # never dereferenced: every call below fails its checks or is empty work
F = ctypes.c_float


def strides(*s):
    return (ctypes.c_int64 * len(s))(*s)


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(binding.LIB_PATH):
        import __graft_entry__
        __graft_entry__.build()
    return binding.lib()


def test_causal_conv_checks(lib):
    base = dict(x=FAKE, dt=1, xs=None, w=FAKE, b=FAKE, act=1, S0=FAKE, S=FAKE, st=None, ln=None, y=P(8192), B=2, H=3, T=40, d=64, K=4,
                stream=None)
    call = lambda **kw: lib.sdm_causal_conv_forward(*dict(base, **kw).values())  # noqa: E731
    for n in ("x", "w", "y"):
        assert call(**{n: None}) == 1, n
    for n in ("w", "b", "S0", "S", "y"):
        assert call(**{n: P(4100)}) == 4, n
    assert call(x=P(4097)) == 4                               # x: its elements' alignment
    assert call(ln=P(4098)) == 4
    assert call(dt=2) == 3 and call(act=2) == 3
    assert call(T=-1) == 2 and call(d=0) == 2 and call(K=0) == 2
    assert call(K=1) == 5 and call(K=9) == 5
    assert call(d=1 << 23, H=2) == 5 and call(B=1 << 20, T=1 << 20) == 5 and call(B=1 << 40) == 5 and call(T=1 << 62) == 5
    assert call(xs=strides(-1, 0, 64)) == 2
    assert call(xs=strides(1 << 60, 1 << 60, 64)) == 5
    assert call(y=FAKE) == 2                                   # y is x
    assert call(S0=P(8192)) == 2 and call(S=P(8192)) == 2
    assert call(B=0, x=None, w=None, y=None) == 0 and call(H=0, x=None, w=None, y=None) == 0
    bwd = dict(dy=FAKE, x=FAKE, dt=1, xs=None, w=FAKE, b=FAKE, act=1, S0=P(1 << 20), dS=P(1 << 21), st=None, ln=None, dx=P(8192), gs=None,
               dw=FAKE, db=FAKE, dS0=P(1 << 22), B=2, H=3, T=40, d=64, K=4, ws=FAKE, wsb=1 << 40, stream=None)
    callb = lambda **kw: lib.sdm_causal_conv_backward(*dict(bwd, **kw).values())  # noqa: E731
    for n in ("dy", "x", "w", "dx", "dw"):
        assert callb(**{n: None}) == 1, n
    for n in ("dy", "w", "b", "S0", "dS", "dw", "db", "dS0"):
        assert callb(**{n: P(4100)}) == 4, n
    assert callb(dx=P(8193)) == 4
    assert callb(dx=FAKE) == 2 and callb(dS0=P(1 << 21)) == 2 and callb(dS0=P(1 << 20)) == 2 and callb(dS0=P(8192)) == 2
    assert callb(gs=strides(0, 64, 192)) == 2 and callb(gs=strides(40 * 192, 63, 192)) == 2 and callb(gs=strides(40 * 64, 64, 192)) == 2
    assert callb(ws=None) == 7 and callb(wsb=100) == 7
    assert callb(B=0, dy=None, x=None, w=None, dx=None, dw=None) == 0
    n = lib.sdm_causal_conv_backward_workspace_bytes
    assert n(0, 1, 1, 1, 4) == 0 and n(1, 1, 1, 1, 9) == -1 and n(1, 1, -1, 1, 4) == -1 and n(1 << 31, 1 << 31, 1 << 31, 1 << 31, 4) == -1
    assert n(2, 3, 40, 64, 4) > 0
    with pytest.raises(ValueError):
        binding.sdm_causal_conv_backward_workspace_bytes(1, 1, 1, 1, 1)


SCAN = dict(x=FAKE, dt=FAKE, z=FAKE, Bm=FAKE, Cm=FAKE, ty=1, s=None, A=FAKE, D=FAKE, bias=FAKE, sp=1, S0=FAKE, S=FAKE, st=None, ln=None,
            y=P(8192), B=2, T=300, Dn=128, G=2, N=16, ws=FAKE, wsb=1 << 40, stream=None)


def test_selective_scan_checks(lib):
    call = lambda **kw: lib.sdm_selective_scan_forward(*dict(SCAN, **kw).values())  # noqa: E731
    for n in ("x", "dt", "Bm", "Cm", "A", "y"):
        assert call(**{n: None}) == 1, n
    for n in ("x", "dt", "z", "Bm", "Cm"):
        assert call(**{n: P(4097)}) == 4, n
        assert call(**{n: P(4098), "ty": 0}) == 4, n
    for n in ("A", "D", "bias", "S0", "S", "y"):
        assert call(**{n: P(4100)}) == 4, n
    assert call(ln=P(4098)) == 4
    assert call(ty=2) == 3 and call(ty=-1) == 3
    assert call(T=-1) == 2 and call(N=0) == 2 and call(G=0) == 2 and call(G=3) == 2
    assert call(N=65) == 5 and call(Dn=1 << 21) == 5 and call(B=1 << 21) == 5 and call(s=strides(*[1 << 26] * 12)) == 5 and call(B=1 << 62) == 5 and call(T=1 << 40) == 5
    for k in range(12):
        bad = [300 * 128, 128] * 3 + [300 * 32, 32, 16] * 2
        bad[k] = -bad[k]
        assert call(s=strides(*bad)) == 2, k
        bad[k] = 1 << 60
        assert call(s=strides(*bad)) == 5, k
    for n in ("x", "dt", "z", "Bm", "Cm", "S0", "S"):
        assert call(**{n: P(8192)}) == 2, n                    # y is an input or the state
    assert call(ws=None) == 7 and call(wsb=64) == 7 and call(ws=P(4100)) == 4
    assert call(B=0, x=None, dt=None, Bm=None, Cm=None, A=None, y=None) == 0
    n = lib.sdm_selective_scan_workspace_bytes
    assert n(2, 1, 128, 1, 16) == 0 and n(0, 300, 128, 1, 16) == 0 and n(2, 300, 128, 3, 16) == -1 and n(2, 300, 128, 1, 65) == -1
    assert n(1 << 31, 1 << 31, 1 << 20, 1, 64) == -1
    for f in (binding.sdm_selective_scan_workspace_bytes, binding.sdm_selective_scan_backward_workspace_bytes):
        with pytest.raises(ValueError):
            f(2, 300, 128, 3, 16)


def test_selective_scan_backward_checks(lib):
    far = {k: P(1 << 20 + i) for i, k in enumerate(("dx", "ddt", "dz", "dB", "dC"))}
    base = dict(dy=FAKE, x=FAKE, dt=FAKE, z=FAKE, Bm=FAKE, Cm=FAKE, ty=1, s=None, A=FAKE, D=FAKE, bias=FAKE, sp=1, S0=FAKE, dS=FAKE,
                st=None, ln=None, dx=far["dx"], ddt=far["ddt"], dz=far["dz"], dA=FAKE, dB=far["dB"], dC=far["dC"], dD=FAKE, db=FAKE,
                dS0=FAKE, B=2, T=300, Dn=128, G=2, N=16, ws=FAKE, wsb=1 << 40, stream=None)
    call = lambda **kw: lib.sdm_selective_scan_backward(*dict(base, **kw).values())  # noqa: E731
    for n in ("dy", "x", "dt", "Bm", "Cm", "A", "dx", "ddt", "dz", "dA", "dB", "dC"):
        assert call(**{n: None}) == 1, n
    for n in ("dx", "ddt", "dz", "dA", "dB", "dC", "dD", "db", "dS0", "A", "S0", "dS"):
        assert call(**{n: P(4100)}) == 4, n
    assert call(dy=P(4097)) == 4
    assert call(ty=3) == 3 and call(N=0) == 2 and call(N=80) == 5
    assert call(s=strides(*[300 * 128, 128] * 3, *[300 * 32, 32, 16] * 2, -1, 128)) == 2
    assert call(T=1 << 27) == 5 and call(Dn=1 << 20, G=1 << 18) == 5 and call(B=1 << 62, T=1 << 62) == 5
    for n in far:
        assert call(**{n: FAKE}) == 2, n
    assert call(ws=None) == 7 and call(wsb=1 << 10) == 7
    assert call(B=0, dy=None, x=None, dA=None) == 0
    n = lib.sdm_selective_scan_backward_workspace_bytes
    assert n(0, 300, 128, 1, 16) == 0 and n(2, 300, 128, 1, 0) == -1 and n(2, 1 << 27, 128, 1, 16) == -1 and n(2, 300, 128, 2, 16) > 0


def test_layer_norm_checks(lib):
    x, r, h, y = P(4096), P(8192), P(12288), P(16384)
    base = dict(x=x, xd=1, r=r, h=h, hd=1, g=FAKE, b=FAKE, eps=F(1e-5), rows=4, d=256, y=y, yd=2, s=FAKE, grp=128, st=None)
    call = lambda **kw: lib.sdm_residual_layer_norm(*dict(base, **kw).values())  # noqa: E731
    assert call(xd=2) == 3 and call(hd=2) == 3 and call(yd=3) == 3
    assert call(rows=-1) == 2 and call(d=0) == 2 and call(eps=F(-1.0)) == 2 and call(yd=1) == 2
    assert call(d=16640) == 5 and call(grp=96) == 5
    for n in ("x", "g", "y", "s"):
        assert call(**{n: None}) == 1, n
    for n in ("x", "g", "b", "y", "s"):
        assert call(**{n: P(4100)}) == 4, n
    assert call(y=x) == 2 and call(y=h) == 2 and call(h=x, xd=0) == 2
    assert call(rows=0, x=None, r=None, h=None, g=None, b=None, y=None, s=None) == 0
    bwd = dict(dy=x, dh=r, gd=1, h=h, hd=1, g=FAKE, eps=F(1e-5), rows=4, d=256, dx=y, dg=FAKE, db=FAKE, ws=FAKE, wsb=1 << 30, st=None)
    callb = lambda **kw: lib.sdm_residual_layer_norm_backward(*dict(bwd, **kw).values())  # noqa: E731
    for n in ("dy", "h", "g", "dx", "dg"):
        assert callb(**{n: None}) == 1, n
    assert callb(gd=2) == 3 and callb(dh=P(4100)) == 4 and callb(db=P(4100)) == 4 and callb(dx=h, hd=0) == 2
    rms, ln = lib.sdm_residual_norm_backward_workspace_bytes, lib.sdm_residual_layer_norm_backward_workspace_bytes
    assert ln(300, 256) == 2 * rms(300, 256) and ln(0, 64) == 0 and ln(5, 16385) == -1
    assert callb(ws=None) == 7 and callb(wsb=2 * 256 * 4 - 1) == 7
    assert callb(rows=0, dy=None, h=None, dx=None, dg=None, db=None) == 0


def test_binding_refuses_cpu_tensors(lib):
    import torch
    x, w, s = torch.zeros(1, 4, 8), torch.zeros(8, 4), torch.zeros(1, 4, 2)
    for call in (lambda: binding.sdm_causal_conv_forward(x, w), lambda: binding.sdm_causal_conv_backward(x, x, w),
                 lambda: binding.sdm_selective_scan_forward(x, x, torch.zeros(8, 2), s, s),
                 lambda: binding.sdm_selective_scan_backward(x, x, x, torch.zeros(8, 2), s, s),
                 lambda: binding.sdm_residual_layer_norm(x, torch.ones(8)),
                 lambda: binding.sdm_residual_layer_norm_backward(x, x, torch.ones(8))):
        with pytest.raises(ValueError):
            call()
