"""The short causal convolution and its gradients against 64 bits.

Tolerances count roundings of half a step (2^-24 in fp32, 2^-8 for outputs in bf16). z: K products and
sums, so (K + 1) of the terms' magnitudes. The sigmoid: its argument, rounded, is off by 1.25 half
steps of |z|, the exponential and the reciprocal by two each; the products by one each, so silu and its derivative
are off by (3 |z| + 14) half steps of their terms, and by 1.1 and 0.6 times what z is off by. The weights' gradient is
a chain of at most 64 sums a tile at these sizes, and 64-bit sums over the tiles.
"""
import pytest
import torch

import sparse_memory_linear_amd as sdm

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
BF, F32 = torch.bfloat16, torch.float32
HALF = {BF: 2.0 ** -8, F32: 2.0 ** -24}
U = 2.0 ** -24


def make(B, H, T, d, K, dtype, seed, state=True):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    p = {"x": r(B, H, T, d).to(dtype), "w": r(H, d, K), "bias": r(H, d), "dy": r(B, H, T, d).to(dtype),
         "S0": r(B, H, K - 1, d).to(dtype) if state else None, "dS": r(B, H, K - 1, d).to(dtype) if state else None}
    return p


def reference(p, act, start=None, lengths=None):
    """All results and their tolerances, by loops over tokens and taps in 64 bits."""
    f = lambda t: t.double()  # noqa: E731
    x, w, bias, dy = f(p["x"]), f(p["w"]), f(p["bias"]), f(p["dy"])
    B, H, T, d = x.shape
    K = w.shape[-1]
    half = HALF[p["x"].dtype]
    zero = torch.zeros(B, H, K - 1, d, dtype=torch.float64)
    S0 = f(p["S0"]) if p["S0"] is not None else zero
    dS = f(p["dS"]) if p["dS"] is not None else zero
    got = {k: torch.zeros_like(v) for k, v in (("y", x), ("S", S0), ("dx", x), ("dw", w), ("dbias", bias), ("dS0", S0))}
    tol = {k: torch.zeros_like(v) for k, v in got.items()}
    for b in range(B):
        n = T if lengths is None else max(0, min(T, int(lengths[b])))
        begin = [bool(start[b, t]) if start is not None else False for t in range(n)]
        seen = lambda t: (S0[b, :, t + K - 1] if t < 0 else x[b, :, t])  # noqa: E731
        first = -K + 1
        firsts = []
        for t in range(n):
            first = t if begin[t] else first
            firsts.append(first)
        for t in range(n):
            z, mag = bias.clone(), bias.abs()
            taps = [(j, t - K + 1 + j) for j in range(K) if t - K + 1 + j >= firsts[t]]
            for j, s in taps:
                z = z + w[:, :, j] * seen(s)
                mag = mag + (w[:, :, j] * seen(s)).abs()
            ez = (K + 1) * U * mag
            if act == "silu":
                sg = torch.sigmoid(z)
                y, dv = z * sg, sg * (1 + z * (1 - sg))
                ey = 1.1 * ez + (3 * z.abs() + 14) * U * y.abs()
                ed = 0.6 * ez + (3 * z.abs() + 14) * U * sg * (1 + z.abs())
            else:
                y, dv, ey, ed = z, torch.ones_like(z), ez, torch.zeros_like(z)
            got["y"][b, :, t] = y
            tol["y"][b, :, t] = ey + half * y.abs()
            dz, edz = dy[b, :, t] * dv, dy[b, :, t].abs() * (ed + 2 * U * dv.abs())
            got["dbias"] += dz
            tol["dbias"] += edz + 67 * U * dz.abs()
            for j, s in taps:
                into, row = (("dS0", s + K - 1) if s < 0 else ("dx", s))
                got[into][b, :, row] += w[:, :, j] * dz
                tol[into][b, :, row] += w[:, :, j].abs() * (edz + (K + 2) * U * dz.abs())
                got["dw"][:, :, j] += dz * seen(s)
                tol["dw"][:, :, j] += (edz + 67 * U * dz.abs()) * seen(s).abs()
        for m in range(K - 1):
            s = n - (K - 1) + m
            if s >= (firsts[-1] if n else -K + 1):
                got["S"][b, :, m] = seen(s)
                into, row = (("dS0", s + K - 1) if s < 0 else ("dx", s))
                got[into][b, :, row] += dS[b, :, m]
                tol[into][b, :, row] += (K + 2) * U * dS[b, :, m].abs()
    for k in ("dx", "dS0"):
        tol[k] += half * (got[k].abs() + tol[k])
    for k in ("dw", "dbias"):
        tol[k] += U * got[k].abs()
    return got, tol


def run(p, act, start=None, lengths=None, x=None, **kw):
    c = {k: None if v is None else v.to(DEV) for k, v in p.items()}
    x = c["x"] if x is None else x
    kw.update(start=None if start is None else start.to(DEV), lengths=None if lengths is None else lengths.to(DEV))
    y, S = sdm.sdm_causal_conv_forward(x, c["w"], c["bias"], act, c["S0"], **kw)
    got = sdm.sdm_causal_conv_backward(c["dy"], x, c["w"], c["bias"], act, c["S0"], c["dS"], **kw)
    return {"y": y, "S": S, **got}


def check(got, want, tol):
    for k, w in want.items():
        g = got[k].cpu().double().reshape(w.shape)
        bad = ~((g - w).abs() <= tol[k] + 1e-37)
        assert not bad.any(), (k, int(bad.sum()), float((g - w).abs().max()))


@pytest.mark.parametrize("act", ["silu", None])
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("B,H,T,d,K", [(1, 1, 1, 1, 2), (2, 1, 1, 64, 4), (1, 3, 2, 7, 3), (2, 2, 3, 8, 8), (1, 1, 5, 12, 8),
                                       (2, 1, 31, 20, 5), (1, 2, 33, 16, 4), (3, 1, 67, 5, 4), (1, 4, 130, 24, 2), (2, 1, 65, 72, 6),
                                       (1, 1, 200, 9, 7)])
def test_against_64_bits(B, H, T, d, K, dtype, act):
    for state in (True, False):
        p = make(B, H, T, d, K, dtype, B + T + d + K, state)
        check(run(p, act), *reference(p, act))


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("T,K,d", [(1, 4, 8), (3, 8, 8), (70, 4, 16), (131, 3, 5), (64, 8, 12)])
def test_packed_and_padded(T, K, d, dtype):
    B, H = 5, 2
    g = torch.Generator().manual_seed(T)
    p = make(B, H, T, d, K, dtype, T + K)
    start = (torch.rand((B, T), generator=g) < 0.15).to(torch.uint8) * 3
    start[0] = 0
    start[1] = 1                      # every token for itself
    start[2, 0] = 1
    start[3, -1] = 1
    lengths = torch.tensor([T, T // 2, 0, -3, T + 9], dtype=torch.int32)
    check(run(p, "silu", start), *reference(p, "silu", start))
    check(run(p, "silu", start.bool()), *reference(p, "silu", start))
    check(run(p, "silu", None, lengths), *reference(p, "silu", None, lengths))
    want, tol = reference(p, "silu", start, lengths)
    for b in range(B):  # what is behind the last token is not looked at
        n = max(0, min(T, int(lengths[b])))
        p["x"][b, :, n:] = float("nan")
        p["dy"][b, :, n:] = float("inf")
    check(run(p, "silu", start, lengths), want, tol)


def test_a_sequence_ends_with_its_infinities():
    p = make(1, 2, 60, 8, 4, F32, 3)
    start = torch.zeros((1, 60), dtype=torch.uint8)
    start[0, [20, 40]] = 1
    want, tol = reference(p, "silu", start)
    p["x"][0, :, 39] = float("inf")
    p["dy"][0, :, 20] = float("nan")
    got = run(p, "silu", start)
    for k in ("y", "dx"):
        e = (got[k].cpu().double() - want[k]).abs() <= tol[k] + 1e-37
        assert e[:, :, :20].all() and e[:, :, 40:].all(), k
    for k in ("S", "dS0"):
        assert ((got[k].cpu().double() - want[k]).abs() <= tol[k] + 1e-37).all(), k


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("d", [16, 13])
def test_strides(d, dtype):
    """Heads out of a projection, a part of a wider one at an odd offset, and gradients written into one."""
    B, H, T, K = 2, 3, 40, 4
    p = make(B, H, T, d, K, dtype, d)
    want, tol = reference(p, "silu")
    heads = p["x"].transpose(1, 2).contiguous().to(DEV).transpose(1, 2)  # [B, T, H, d] in memory
    got = run(p, "silu", x=heads)
    assert got["dx"].stride() == heads.stride()
    check(got, want, tol)
    for offset in (8, 3):
        wide = torch.full((B, T, H * d + 11), float("nan"), dtype=dtype, device=DEV)
        part = wide[..., offset:offset + H * d].view(B, T, H, d).transpose(1, 2)
        part.copy_(p["x"])
        check(run(p, "silu", x=part), want, tol)
        grad = torch.full_like(wide, 7.0)
        dx = grad[..., offset:offset + H * d].view(B, T, H, d).transpose(1, 2)
        c = {k: v.to(DEV) for k, v in p.items()}
        got = sdm.sdm_causal_conv_backward(c["dy"], part, c["w"], c["bias"], "silu", c["S0"], c["dS"], out={"dx": dx})
        assert got["dx"] is dx
        check(got, {k: want[k] for k in got}, tol)
        assert (grad[..., :offset] == 7).all() and (grad[..., offset + H * d:] == 7).all()
    one = p["x"][:1].to(DEV).expand(B, H, T, d)  # one input for all sequences
    q = dict(p, x=p["x"][:1].expand(B, H, T, d).contiguous())
    check(run(p, "silu", x=one), *reference(q, "silu"))


def test_three_dimensions_are_one_head():
    p = make(2, 1, 19, 24, 4, BF, 0)
    flat = {k: (v[0] if k in ("w", "bias") else v[:, 0]).contiguous() for k, v in p.items()}
    a, b = run(p, "silu"), run(flat, "silu")
    for k in a:
        assert torch.equal(a[k].reshape(b[k].shape), b[k]), k
    assert b["y"].shape == (2, 19, 24) and b["dw"].shape == (24, 4) and b["dS0"].shape == (2, 3, 24)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_a_sequence_in_pieces(dtype):
    """Prompts and single tokens with the state in place give what one call gives, bit for bit."""
    p = make(2, 2, 50, 24, 5, dtype, 1)
    c = {k: v.to(DEV) for k, v in p.items()}
    whole, last = sdm.sdm_causal_conv_forward(c["x"], c["w"], c["bias"], "silu", c["S0"])
    S, ys, t = c["S0"].clone(), [], 0
    for n in (20, 1, 1, 2, 3, 1, 4, 18):
        y, S2 = sdm.sdm_causal_conv_forward(c["x"][:, :, t:t + n], c["w"], c["bias"], "silu", S, S)
        assert S2 is S
        ys.append(y)
        t += n
    assert torch.equal(torch.cat(ys, 2), whole) and torch.equal(S, last)
    dS, dxs, dw = c["dS"], [], 0
    full = sdm.sdm_causal_conv_backward(c["dy"], c["x"], c["w"], c["bias"], "silu", c["S0"], dS)
    cut = 33
    _, mid = sdm.sdm_causal_conv_forward(c["x"][:, :, :cut], c["w"], c["bias"], "silu", c["S0"])
    b = sdm.sdm_causal_conv_backward(c["dy"][:, :, cut:].contiguous(), c["x"][:, :, cut:], c["w"], c["bias"], "silu", mid, dS)
    a = sdm.sdm_causal_conv_backward(c["dy"][:, :, :cut].contiguous(), c["x"][:, :, :cut], c["w"], c["bias"], "silu", c["S0"], b["dS0"])
    # the gradient that passes the cut is rounded there
    want, tol = reference(p, "silu")
    got = {"dx": torch.cat([a["dx"], b["dx"]], 2), "dw": a["dw"] + b["dw"], "dbias": a["dbias"] + b["dbias"], "dS0": a["dS0"]}
    for k in got:
        e = (got[k].cpu().double() - want[k]).abs()
        assert (e <= 2 * tol[k] + HALF[dtype] * full["dx"].abs().max().item() + 1e-37).all(), k


def test_no_tokens_and_no_sequences():
    p = make(2, 2, 4, 8, 4, BF, 0)
    c = {k: v.to(DEV) for k, v in p.items()}
    x = c["x"][:, :, :0]
    y, S = sdm.sdm_causal_conv_forward(x, c["w"], c["bias"], "silu", c["S0"])
    assert y.shape == (2, 2, 0, 8) and torch.equal(S, c["S0"])
    got = sdm.sdm_causal_conv_backward(c["dy"][:, :, :0].contiguous(), x, c["w"], c["bias"], "silu", c["S0"], c["dS"])
    assert torch.equal(got["dS0"], c["dS"]) and (got["dw"] == 0).all() and (got["dbias"] == 0).all()
    y, S = sdm.sdm_causal_conv_forward(x, c["w"])
    assert (S == 0).all()
    e = c["x"][:0]
    y, S = sdm.sdm_causal_conv_forward(e, c["w"])
    got = sdm.sdm_causal_conv_backward(e.contiguous(), e, c["w"])
    assert y.shape == (0, 2, 4, 8) and S.shape == (0, 2, 3, 8) and (got["dw"] == 0).all()


def test_gradients_against_differences():
    """d/ds of <dy, y> + <dS, S> along a random direction, by a central difference of the forward call in fp32:
    its own error is some 2^-23 of the sum's magnitude over the step, and the third derivative's share."""
    p = make(2, 2, 30, 8, 4, F32, 9)
    c = {k: v.to(DEV) for k, v in p.items()}
    got = sdm.sdm_causal_conv_backward(c["dy"], c["x"], c["w"], c["bias"], "silu", c["S0"], c["dS"])
    g = torch.Generator().manual_seed(3)
    for name in ("x", "w", "bias", "S0"):
        v = torch.randn(c[name].shape, generator=g).to(DEV)
        h = 2.0 ** -6

        def loss(s):
            q = dict(c, **{name: c[name] + s * v})
            y, S = sdm.sdm_causal_conv_forward(q["x"], q["w"], q["bias"], "silu", q["S0"])
            return float((y.double() * c["dy"].double()).sum() + (S.double() * c["dS"].double()).sum())

        want = float((got["d" + name].double() * v.double()).sum())
        size = float((got["d" + name].double() * v.double()).abs().sum())
        assert abs((loss(h) - loss(-h)) / (2 * h) - want) <= 2e-3 * size, name


def test_far_rows():
    """Offsets beyond 2^31 elements of x: sequences a long way apart."""
    B, T, d, K = 2, 5, 16, 4
    p = make(B, 1, T, d, K, BF, 4)
    far = torch.zeros((1 << 31) + 4096, dtype=BF, device=DEV)
    x = far.as_strided((B, 1, T, d), ((1 << 31) + 64, 0, d, 1))
    x.copy_(p["x"])
    check(run(p, "silu", x=x), *reference(p, "silu"))


@pytest.mark.parametrize("break_it", [
    lambda c: dict(x=c["x"].transpose(2, 3)), lambda c: dict(w=c["w"].to(BF)), lambda c: dict(w=c["w"][:, :4]),
    lambda c: dict(bias=c["bias"][:1]), lambda c: dict(S0=c["S0"].float()), lambda c: dict(S0=c["S0"][:, :, :2]),
    lambda c: dict(act="gelu"), lambda c: dict(w=c["w"][..., :1]), lambda c: dict(x=c["x"].half()),
    lambda c: dict(start=torch.zeros((2, 5), device=DEV)), lambda c: dict(lengths=torch.zeros(2, dtype=torch.int64, device=DEV)),
    lambda c: dict(x=c["x"].cpu()), lambda c: dict(x=c["x"][0, 0])])
def test_refusals(break_it):
    c = {k: v.to(DEV) for k, v in make(2, 2, 6, 8, 4, BF, 0).items()}
    good = dict(x=c["x"], w=c["w"], bias=c["bias"], act="silu", S0=c["S0"])
    sdm.sdm_causal_conv_forward(**good)
    with pytest.raises(ValueError):
        sdm.sdm_causal_conv_forward(**dict(good, **break_it(c)))


def test_refusals_of_the_library():
    c = {k: v.to(DEV) for k, v in make(2, 2, 6, 8, 4, BF, 0).items()}
    with pytest.raises(sdm.SdmError):
        sdm.sdm_causal_conv_forward(c["x"], torch.zeros((2, 8, 9), device=DEV))
    with pytest.raises(sdm.SdmError):
        sdm.sdm_causal_conv_forward(c["x"], c["w"], y=c["x"])
    with pytest.raises(sdm.SdmError):  # rows of dx over each other
        sdm.sdm_causal_conv_backward(c["dy"], c["x"], c["w"], out={"dx": c["x"].new_zeros((2, 1, 6, 8)).expand(2, 2, 6, 8)})
    with pytest.raises(ValueError):
        sdm.sdm_causal_conv_backward(c["dy"], c["x"], c["w"], out={"dS": c["dS"]})
