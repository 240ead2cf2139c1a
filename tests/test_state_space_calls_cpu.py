"""Host-side checks (no GPU) of calls at the edges of what the state-space layer's entry points take: no tokens, the
largest sizes, tensors over each other. Every call here is refused before any launch."""
import ctypes
import os

import pytest

from sparse_memory_linear_amd import binding

P = ctypes.c_void_p
NULL, SHAPE, UNSUPPORTED, WORKSPACE = 1, 2, 5, 7


def at(k):
    """Aligned addresses far from each other; never dereferenced."""
    return P((k + 1) << 40)


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(binding.LIB_PATH):
        import __graft_entry__
        __graft_entry__.build()
    return binding.lib()


CONV_BWD = dict(dy=at(0), x=at(1), dtype=1, xs=None, w=at(2), bias=at(3), act=1, S0=at(4), dS=at(5), start=None, lengths=None,
                dx=at(6), gs=None, dw=at(7), dbias=at(8), dS0=at(9), B=2, H=2, T=5, d=8, K=4, ws=None, bytes=0, stream=None)


def conv_bwd(lib, **kw):
    return lib.sdm_causal_conv_backward(*dict(CONV_BWD, **kw).values())


def test_convolution_backward_of_no_tokens(lib):
    """Contiguous tensors (no strides given) of no tokens hold no element twice: what is missing is the workspace."""
    for B, H in ((1, 1), (2, 1), (1, 2), (2, 2), (300, 7)):
        assert conv_bwd(lib, B=B, H=H, T=0, dy=None, x=None, dx=None) == WORKSPACE, (B, H)
        assert conv_bwd(lib, B=B, H=H, T=0, dy=None, x=None, dx=None, dS0=CONV_BWD["dS"]) == WORKSPACE, (B, H)
    zero = (ctypes.c_int64 * 3)(0, 0, 8)
    assert conv_bwd(lib, T=0, gs=zero) == WORKSPACE
    assert conv_bwd(lib, T=1, gs=zero) == SHAPE and conv_bwd(lib, T=1) == WORKSPACE


def test_selective_scan_backward_at_its_largest(lib):
    """dB and dC are added by 32 threads a token, group and tile of 16 states, in workgroups of 256: with those rounded up, the
    launch has to stay below 2^32 threads, or it would fail behind the passes in front of it."""
    n = lib.sdm_selective_scan_backward_workspace_bytes
    for B, T, D, G, N in ((1, 1 << 27, 64, 1, 16), (2, 1 << 26, 64, 1, 16), (1, 1 << 26, 64, 2, 16), (1, 1 << 25, 64, 1, 64)):
        per = B * G * -(-N // 16)
        fits = [T - k for k in range(0, 12) if -(-per * (T - k) * 32 // 256) * 256 < 1 << 32]
        assert fits and all(n(B, t, D, G, N) > 0 for t in fits), (B, T)
        assert all(n(B, T - k, D, G, N) == -1 for k in range(0, 12) if T - k not in fits), (B, T)


SCAN_IN = ("x", "dt", "z", "Bm", "Cm", "A", "D", "bias")
SCAN_BWD = dict(dy=at(0), x=at(1), dt=at(2), z=at(3), Bm=at(4), Cm=at(5), dtype=1, strides=None, A=at(6), D=at(7), bias=at(8), softplus=1,
                S0=at(9), dS=at(10), start=None, lengths=None, dx=at(11), ddt=at(12), dz=at(13), dA=at(14), dB=at(15), dC=at(16), dD=at(17),
                dbias=at(18), dS0=at(19), B=2, T=300, Dn=128, G=2, N=16, ws=at(20), bytes=1 << 40, stream=None)


def test_selective_scan_gradients_over_each_other(lib):
    """Two gradients at one address, or one at that of an input which is read beside it."""
    call = lambda **kw: lib.sdm_selective_scan_backward(*dict(SCAN_BWD, **kw).values())  # noqa: E731
    outs = ("dx", "ddt", "dz", "dA", "dB", "dC", "dD", "dbias", "dS0")
    for i, a in enumerate(outs):
        for b in outs[:i]:
            assert call(**{a: SCAN_BWD[b]}) == SHAPE, (a, b)
    for a in ("dx", "ddt", "dz", "dB", "dC", "dS0"):
        for b in ("dy", *SCAN_IN):
            assert call(**{a: SCAN_BWD[b]}) == SHAPE, (a, b)
    for a, b in (("dD", "dA"), ("dbias", "dD"), ("dS0", "dA")):  # without tokens too
        assert call(T=0, **{a: SCAN_BWD[b]}) == SHAPE, (a, b)
    assert call(dS0=SCAN_BWD["dS"], ws=None) == WORKSPACE and call(dz=SCAN_BWD["x"], z=None, ws=None) == WORKSPACE


def test_states_over_inputs(lib):
    """The state behind the last token may be written over S0, and over nothing that the call reads."""
    conv = dict(x=at(0), dtype=1, xs=None, w=at(1), bias=at(2), act=1, S0=at(3), S=at(4), start=None, lengths=None, y=at(5), B=2, H=2, T=5, d=8,
                K=4, stream=None)
    for b in ("x", "w", "bias"):
        assert lib.sdm_causal_conv_forward(*dict(conv, S=conv[b]).values()) == SHAPE, b
    scan = {k: v for k, v in SCAN_BWD.items() if k in (*SCAN_IN, "dtype", "strides", "softplus", "S0", "start", "lengths")}
    names = ("x", "dt", "z", "Bm", "Cm", "dtype", "strides", "A", "D", "bias", "softplus", "S0", "S", "start", "lengths", "y")
    scan.update(S=at(10), y=at(11))
    tail = (2, 300, 128, 2, 16, at(20), 1 << 40, None)
    for b in SCAN_IN:
        assert lib.sdm_selective_scan_forward(*(dict(scan, S=scan[b])[n] for n in names), *tail) == SHAPE, b


def test_convolution_gradients_over_each_other(lib):
    big = dict(ws=at(10), bytes=1 << 40)
    outs = ("dx", "dw", "dbias", "dS0")
    for i, a in enumerate(outs):
        for b in outs[:i]:
            assert conv_bwd(lib, **{a: CONV_BWD[b]}, **big) == SHAPE, (a, b)
    for a in ("dx", "dS0"):
        for b in ("dy", "x", "w", "bias", "S0", "dS"):
            assert conv_bwd(lib, **{a: CONV_BWD[b]}, **big) == SHAPE, (a, b)
    assert conv_bwd(lib, T=0, dw=CONV_BWD["dbias"], **big) == SHAPE and conv_bwd(lib, T=0, dw=CONV_BWD["dS0"], **big) == SHAPE


def test_layer_norm_outputs_over_each_other(lib):
    f = ctypes.c_float
    norm = dict(x=at(0), xd=1, res=at(1), h=at(2), hd=1, gamma=at(3), bias=at(4), eps=f(1e-5), rows=4, d=256, y=at(5), yd=2, scale=at(6),
                group=128, stream=None)
    for a, b in (("y", "gamma"), ("y", "bias"), ("h", "gamma"), ("h", "bias"), ("scale", "gamma"), ("scale", "bias"), ("scale", "x"),
                 ("scale", "res"), ("scale", "y"), ("scale", "h")):
        assert lib.sdm_residual_layer_norm(*dict(norm, **{a: norm[b]}).values()) == SHAPE, (a, b)
    back = dict(dy=at(0), dh=at(1), gd=0, h=at(2), hd=0, gamma=at(3), eps=f(1e-5), rows=4, d=256, dx=at(4), dgamma=at(5), dbias=at(6), ws=at(7),
                bytes=1 << 40, stream=None)
    for a, b in (("dgamma", "dbias"), ("dx", "dgamma"), ("dx", "dbias"), ("dx", "gamma")):
        assert lib.sdm_residual_layer_norm_backward(*dict(back, **{a: back[b]}).values()) == SHAPE, (a, b)
    for b in ("dy", "dh", "h"):  # (over a row's own inputs it may be)
        assert lib.sdm_residual_layer_norm_backward(*dict(back, dx=back[b], ws=None).values()) == WORKSPACE, b
