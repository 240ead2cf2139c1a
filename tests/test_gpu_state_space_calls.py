"""Calls at the edges of what the state-space layer's entry points take, on the GPU."""
import math

import pytest
import torch

import sparse_memory_linear_amd as sdm
from sparse_memory_linear_amd import binding

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
BF, F32 = torch.bfloat16, torch.float32


def gen(seed):
    g = torch.Generator().manual_seed(seed)
    return lambda *s: torch.randn(s, generator=g).to(DEV)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("B,H,d,K", [(2, 2, 8, 4), (3, 1, 5, 2), (1, 4, 12, 8)])
def test_convolution_backward_of_no_tokens(B, H, d, K, dtype):
    """No tokens, no strides given: the state's gradient is passed on, also in place, and the weights' are 0."""
    L, r, p = binding.lib(), gen(1), lambda t: t.data_ptr()  # noqa: E731
    w, S0, dS = r(H, d, K), r(B, H, K - 1, d).to(dtype), r(B, H, K - 1, d).to(dtype)
    want = dS.clone()
    ws = torch.empty(L.sdm_causal_conv_backward_workspace_bytes(B, H, 0, d, K), dtype=torch.uint8, device=DEV)
    for dS0 in (torch.full_like(dS, 7.0), dS):
        dw, db = torch.full_like(w, 7.0), torch.full((H, d), 7.0, device=DEV)
        rc = L.sdm_causal_conv_backward(None, None, int(dtype == BF), None, p(w), None, 1, p(S0), p(dS), None, None, None, None, p(dw), p(db),
                                        p(dS0), B, H, 0, d, K, p(ws), ws.numel(), torch.cuda.current_stream().cuda_stream)
        assert rc == 0, L.sdm_last_error()
        assert torch.equal(dS0, want) and (dw == 0).all() and (db == 0).all()


def test_sums_of_many_like_terms():
    """So many sequences that none has to be cut, of 8192 tokens all alike: a sum of n like terms in one chain of fp32 is off
    by up to n / 2 half steps (each addition by half a step of the sum so far), and no more than 1024 may be in one. The terms
    themselves are off by 64 half steps at most (decays of 0.6 off by 4, 2.5 times over in a state and its gradient each)."""
    B, T, c = 4096, 8192, 0.9
    full = lambda v: torch.full((1, 1, 1), v, device=DEV)  # noqa: E731
    x, dt, dy, Bm, Cm = (full(v).expand(B, T, 1) for v in (1.0, 0.5, c, 0.7, 0.3))
    A, D = torch.full((1, 1), -1.0, device=DEV), torch.zeros(1, device=DEV)
    got = sdm.sdm_selective_scan_backward(dy, x, dt, A, Bm, Cm, D, softplus=False)
    f = lambda t: float(t.flatten()[0])  # noqa: E731  (as fp32 holds them)
    c, b, k = f(dy), f(Bm), f(Cm)
    a, h, hs = math.exp(-0.5), 0.0, [0.0]
    for _ in range(T):
        h = a * h + 0.5 * b
        hs.append(h)
    q, dA, dbias = 0.0, 0.0, 0.0
    for t in reversed(range(T)):
        q += c * k
        w = q * a * hs[t]
        dA += 0.5 * w
        dbias += q * b - w
        q *= a
    # the sums, and the magnitudes of what their terms are made of (a step's: w and q b, w in all 2 dA)
    for name, want, size in (("dD", c * T, c * T), ("dA", dA, dA), ("ddt_bias", dbias, dbias + 4 * dA)):
        e = abs(float(got[name].flatten()[0].double()) / B - want)
        assert e <= (1024 / 2 * want + 64 * size) * 2.0 ** -24, (name, e / want)


def test_sums_over_many_channels():
    """The gradients of B and C of 2^17 like channels: 64 are added in a tree (6 half steps of the sum), the 2048 tiles' sums in
    64 bits, rounded once; a term is off by 16 half steps at most (a decay by 4, and its products)."""
    D, x, dt, c, b, k = 1 << 17, 1.0, 0.5, 0.9, 0.7, 0.3
    full = lambda v, n: torch.full((1, 2, n), v, device=DEV)  # noqa: E731
    tx, td, tc, tb, tk = full(x, D), full(dt, D), full(c, D), full(b, 1), full(k, 1)
    got = sdm.sdm_selective_scan_backward(tc, tx, td, torch.full((D, 1), -1.0, device=DEV), tb, tk, softplus=False)
    c, b, k = (float(t.flatten()[0]) for t in (tc, tb, tk))
    a, h1 = math.exp(-dt), dt * b
    h2, g2 = a * h1 + dt * b, c * k
    for name, want in (("dC", (c * h1, c * h2)), ("dB", (dt * (g2 + a * g2), dt * g2))):
        for t in range(2):
            e = abs(float(got[name][0, t, 0].double()) / (D * want[t]) - 1)
            assert e <= (6 + 16 + 1) * 2.0 ** -24, (name, t, e)
