"""The selective state-space scan and its gradients against 64 bits.

Tolerances: every result is a sum of products along paths through the tokens. A path's product passes through at
most T decays, each with some 4 roundings of half a step (the step's product with A, its exponential, the product
with the state, the sum), and some 64 for its ends (the softplus, the activations, the sums over states and
channels), so it is off by (4 T + 64) 2^-24 of the sum of the terms' magnitudes. A decay exp(delta A) is also off by
|delta A| times what delta is off by (up to 20 half steps, for |dt| up to 8, and in a segment's sum of steps a half step a
token): x exp(-x) <= exp(-x/2), so the magnitudes are taken with decays of exp(delta A / 2). Outputs
add half a step of their type.
"""
import pytest
import torch

import sparse_memory_linear_amd as sdm

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
BF, F32 = torch.bfloat16, torch.float32
HALF = {BF: 2.0 ** -8, F32: 2.0 ** -24}
NAMES = ("x", "dt", "A", "B", "C", "D", "z", "dt_bias", "S0")


def make(B, T, D, G, N, dtype, seed, plain=False):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    return {"x": r(B, T, D).to(dtype), "dt": (r(B, T, D) * 1.5 - 1.0).to(dtype), "A": -torch.exp(0.7 * r(D, N)),
            "B": r(B, T, G, N).to(dtype), "C": r(B, T, G, N).to(dtype), "D": None if plain else r(D),
            "z": None if plain else r(B, T, D).to(dtype), "dt_bias": None if plain else 0.5 * r(D),
            "S0": None if plain else r(B, D, N), "dy": r(B, T, D).to(dtype), "dS": None if plain else r(B, D, N)}


def formulas(p, softplus, keep, go, mags):
    """The results by the formulas; with ``mags`` their terms' magnitudes, and decays of half the exponent."""
    f = (lambda t: t.double().abs()) if mags else (lambda t: t.double())
    B, T, Dd = p["x"].shape
    G, N = p["B"].shape[2:]
    zero = torch.zeros(B, Dd, N, dtype=torch.float64)
    x, Bm, Cm, dy = f(p["x"]), f(p["B"]), f(p["C"]), f(p["dy"])
    A, fA = p["A"].double(), f(p["A"])
    D = f(p["D"]) if p["D"] is not None else torch.zeros(Dd, dtype=torch.float64)
    v = p["dt"].double() + (p["dt_bias"].double() if p["dt_bias"] is not None else 0.0)
    delta = torch.nn.functional.softplus(v) if softplus else v
    delta = delta * keep[..., None]
    h = f(p["S0"]) if p["S0"] is not None else zero
    q = f(p["dS"]) if p["dS"] is not None else zero
    x, dy = x * keep[..., None], dy * keep[..., None]
    Bm, Cm = Bm * keep[..., None, None], Cm * keep[..., None, None]
    spread = lambda m, t: m[:, t].repeat_interleave(Dd // G, 1)  # noqa: E731
    a = [(delta[:, t, :, None] * A * (0.5 if mags else 1.0)).exp() * go[:, t, None, None] for t in range(T)]
    ad = delta.abs() if mags else delta
    hs, y = [h], torch.zeros_like(x)
    for t in range(T):
        h = a[t] * h + (ad[:, t] * x[:, t])[..., None] * spread(Bm, t)
        hs.append(h)
        y[:, t] = (h * spread(Cm, t)).sum(-1)
    y = y + D * x
    if p["z"] is None:
        gate, dgate = torch.ones_like(x), None
    else:
        z = p["z"].double()
        s = torch.sigmoid(z)
        gate, dgate = z * s, s * (1 + z * (1 - s))
        if mags:
            gate, dgate = gate.abs(), s * (1 + z.abs())
        gate = gate * keep[..., None]
    got = {"y": y * gate, "S": h}
    if p["z"] is not None:
        got["dz"] = torch.where(keep[..., None] > 0, dy * y * dgate, 0.0)
    gy = dy * gate
    dx, dd = D * gy, torch.zeros_like(x)
    dA, dB, dC = torch.zeros_like(A), torch.zeros_like(Bm), torch.zeros_like(Cm)
    for t in reversed(range(T)):
        q = q + gy[:, t, :, None] * spread(Cm, t)
        dC[:, t] = (gy[:, t, :, None] * hs[t + 1]).view(B, G, Dd // G, N).sum(2)
        w = q * a[t] * hs[t]
        qb = (q * spread(Bm, t)).sum(-1)
        dd[:, t] = (w * fA).sum(-1) + x[:, t] * qb
        dA += (w * ad[:, t, :, None]).sum(0)
        dx[:, t] += ad[:, t] * qb
        dB[:, t] = (q * (ad[:, t] * x[:, t])[..., None]).view(B, G, Dd // G, N).sum(2)
        q = a[t] * q
    if softplus:
        dd = dd * torch.sigmoid(v)
    dd = dd * keep[..., None]
    on = keep[..., None, None]
    got.update(dx=dx * keep[..., None], ddt=dd, dA=dA, dB=dB * on, dC=dC * on, dD=(gy * x).sum((0, 1)), ddt_bias=dd.sum((0, 1)), dS0=q)
    return got


def reference(p, softplus=True, start=None, lengths=None):
    B, T, _ = p["x"].shape
    n = torch.full((B,), T) if lengths is None else lengths.clamp(0, T)
    keep = (torch.arange(T)[None] < n[:, None]).double()
    go = torch.ones_like(keep)
    if start is not None:
        go = torch.where((start != 0) & (keep > 0), 0.0, 1.0).double()
    p = {k: torch.where(keep.view(B, T, *[1] * (v.dim() - 2)) > 0, v, torch.zeros_like(v)) if k in ("x", "dt", "B", "C", "z", "dy") and v is not None
         else v for k, v in p.items()}
    want, mag = formulas(p, softplus, keep, go, False), formulas(p, softplus, keep, go, True)
    half = HALF[p["x"].dtype]
    tol = {k: (4 * T + 64) * 2.0 ** -24 * mag[k] * 1.01 + (half if k in ("y", "dx", "ddt", "dz") else 2.0 ** -24) * 1.01 * want[k].abs()
           for k in want}
    return want, tol


def run(p, softplus=True, start=None, lengths=None, **over):
    c = {k: None if v is None else v.to(DEV) for k, v in p.items()}
    c.update(over)
    kw = dict(start=None if start is None else start.to(DEV), lengths=None if lengths is None else lengths.to(DEV))
    args = (c["x"], c["dt"], c["A"], c["B"], c["C"], c["D"], c["z"], c["dt_bias"], softplus, c["S0"])
    y, S = sdm.sdm_selective_scan_forward(*args, **kw)
    return {"y": y, "S": S, **sdm.sdm_selective_scan_backward(c["dy"], *args, c["dS"], **kw)}


def check(got, want, tol):
    for k, w in want.items():
        if k not in got:
            assert k == "dz"
            continue
        g = got[k].cpu().double().reshape(w.shape)
        bad = ~((g - w).abs() <= tol[k] + 1e-37)
        assert not bad.any(), (k, int(bad.sum()), float((g - w).abs().max()), float((g - w).abs().norm() / w.norm()))


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("B,T,D,G,N", [(1, 1, 1, 1, 1), (2, 1, 64, 1, 16), (1, 2, 3, 3, 5), (2, 3, 65, 1, 16), (1, 7, 130, 2, 9),
                                       (3, 8, 64, 1, 17), (1, 9, 70, 1, 33), (2, 13, 48, 4, 48), (1, 40, 64, 1, 64), (2, 64, 40, 1, 12),
                                       (1, 65, 64, 1, 16), (2, 131, 96, 2, 20), (1, 200, 36, 1, 7)])
def test_against_64_bits(B, T, D, G, N, dtype):
    for plain in (False, True):
        p = make(B, T, D, G, N, dtype, B + T + D + N, plain)
        check(run(p), *reference(p))


def test_steps_as_given():
    p = make(2, 75, 70, 1, 16, F32, 3)
    p["dt"] = torch.rand(p["dt"].shape, generator=torch.Generator().manual_seed(1)) * 0.5
    p["dt_bias"] = None
    p["dt"][0, 5] = 0.0  # a step of 0 neither writes nor forgets
    check(run(p, False), *reference(p, False))


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("T,D,N", [(1, 64, 16), (1, 70, 40), (6, 10, 3), (43, 70, 16), (43, 64, 40), (150, 70, 16), (203, 64, 30)])
def test_packed_and_padded(T, D, N, dtype):
    B = 5
    g = torch.Generator().manual_seed(T)
    p = make(B, T, D, 1, N, dtype, T + N)
    start = (torch.rand((B, T), generator=g) < 0.04).to(torch.uint8) * 2
    start[0] = 0
    start[1] = 1
    start[2, 0] = 1
    start[3, -1] = 1
    lengths = torch.tensor([T, T // 2, 0, -3, T + 9], dtype=torch.int32)
    check(run(p, True, start), *reference(p, True, start))
    check(run(p, True, start.bool()), *reference(p, True, start))
    check(run(p, True, None, lengths), *reference(p, True, None, lengths))
    want, tol = reference(p, True, start, lengths)
    for b in range(B):  # what is behind the last token is not looked at
        n = max(0, min(T, int(lengths[b])))
        for k, bad in (("x", "nan"), ("dt", "inf"), ("z", "nan"), ("B", "nan"), ("C", "inf"), ("dy", "nan")):
            p[k][b, n:] = float(bad)
    got = run(p, True, start, lengths)
    check(got, want, tol)
    for k in ("y", "dx", "ddt", "dz", "dB", "dC"):
        assert (got[k].cpu()[torch.arange(T)[None] >= lengths[:, None]] == 0).all(), k


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_many_segments(dtype):
    """One narrow sequence: the tokens are cut, sequences begin inside, at and across the cuts, and the end is padding."""
    T, D, N = 900, 24, 8
    p = make(2, T, D, 1, N, dtype, 11)
    start = torch.zeros((2, T), dtype=torch.uint8)
    start[0, [63, 64, 65, 128, 300, 301, 575, 576, 640]] = 1
    lengths = torch.tensor([T, 577], dtype=torch.int32)
    check(run(p, True, start, lengths), *reference(p, True, start, lengths))
    p["dt"] = p["dt"] - 6  # long memories: what the carries bring counts
    check(run(p), *reference(p))


def test_wide_tiles_and_strides():
    """x, z, B and C as parts of projections, dy as a part, at addresses of a single element's alignment."""
    B, T, D, G, N = 2, 77, 72, 2, 16
    for dtype in (BF, F32):
        p = make(B, T, D, G, N, dtype, 5)
        want, tol = reference(p)
        xz = torch.full((B, T, 2 * D + 3), float("nan"), dtype=dtype, device=DEV)
        x, z = xz[..., 1:D + 1], xz[..., D + 2:2 * D + 2]
        low = torch.full((B, T, 7 + 2 * G * N), float("nan"), dtype=dtype, device=DEV)
        Bm, Cm = low[..., 5:5 + G * N].view(B, T, G, N), low[..., 6 + G * N:6 + 2 * G * N].view(B, T, G, N)
        dt = torch.empty((T, B, D), dtype=dtype, device=DEV).transpose(0, 1)  # tokens first
        dy = torch.empty((B, T, D + 1), dtype=dtype, device=DEV)[..., 1:]
        for t, n in ((x, "x"), (z, "z"), (Bm, "B"), (Cm, "C"), (dt, "dt"), (dy, "dy")):
            t.copy_(p[n])
        check(run(p, x=x, z=z, B=Bm, C=Cm, dt=dt, dy=dy), want, tol)
        q = dict(p, B=p["B"][:, :1].expand(B, T, G, N).contiguous())  # one B for all tokens
        check(run(q, B=Bm[:, :1].expand(B, T, G, N)), *reference(q))


def test_groups_of_one_dimension_less():
    p = make(2, 20, 64, 1, 16, BF, 8)
    a = run(p)
    b = run(p, B=p["B"][:, :, 0].contiguous().to(DEV), C=p["C"][:, :, 0].contiguous().to(DEV))
    for k in a:
        assert torch.equal(a[k].reshape(b[k].shape), b[k]), k
    assert b["dB"].shape == (2, 20, 16)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_a_sequence_in_pieces(dtype):
    """A prompt, then single tokens with the state in place; backwards with the gradient of the state passed on."""
    T, cut = 90, 80
    p = make(2, T, 70, 1, 16, dtype, 2)
    want, tol = reference(p)
    c = {k: v.to(DEV) for k, v in p.items()}
    part = lambda a, b: [c[k][:, a:b] for k in ("x", "dt")] + [c["A"]] + [c[k][:, a:b] for k in ("B", "C")] + [c["D"], c["z"][:, a:b], c["dt_bias"], True]  # noqa: E731
    y, S = sdm.sdm_selective_scan_forward(*part(0, cut), c["S0"])
    mid, ys = S.clone(), [y]
    for t in range(cut, T):
        y, S2 = sdm.sdm_selective_scan_forward(*part(t, t + 1), S, S)
        assert S2 is S
        ys.append(y)
    check({"y": torch.cat(ys, 1), "S": S}, {k: want[k] for k in ("y", "S")}, tol)
    b = sdm.sdm_selective_scan_backward(c["dy"][:, cut:], *part(cut, T), mid, c["dS"])
    a = sdm.sdm_selective_scan_backward(c["dy"][:, :cut], *part(0, cut), c["S0"], b["dS0"])
    got = {k: torch.cat([a[k], b[k]], 1) for k in ("dx", "ddt", "dz", "dB", "dC")}
    got.update({k: a[k] + b[k] for k in ("dA", "dD", "ddt_bias")}, dS0=a["dS0"])
    check(got, {k: want[k] for k in got}, tol)


def test_gradient_of_the_state_in_place():
    p = make(2, 70, 64, 1, 16, F32, 6)
    want = run(p)
    c = {k: v.to(DEV) for k, v in p.items()}
    dS = c["dS"].clone()
    got = sdm.sdm_selective_scan_backward(c["dy"], c["x"], c["dt"], c["A"], c["B"], c["C"], c["D"], c["z"], c["dt_bias"], True, c["S0"], dS,
                                          out={"dS0": dS})
    assert got["dS0"] is dS
    for k, v in got.items():
        assert torch.equal(v, want[k]), k


def test_no_tokens_and_no_sequences():
    p = make(2, 4, 70, 1, 16, BF, 0)
    c = {k: v.to(DEV) for k, v in p.items()}
    for lo, hi, dims in ((0, 0, 1), (0, 0, 0)):
        q = {k: (v[:, :0] if dims else v[:0]) if k in ("x", "dt", "B", "C", "z", "dy") else v[:0] if not dims and k in ("S0", "dS") else v
             for k, v in c.items()}
        args = (q["x"], q["dt"], q["A"], q["B"], q["C"], q["D"], q["z"], q["dt_bias"], True, q["S0"])
        y, S = sdm.sdm_selective_scan_forward(*args)
        got = sdm.sdm_selective_scan_backward(q["dy"], *args, q["dS"])
        assert y.shape == q["x"].shape and torch.equal(S, q["S0"]) and torch.equal(got["dS0"], q["dS"])
        for k in ("dA", "dD", "ddt_bias"):
            assert (got[k] == 0).all(), k


def test_a_channel_keeps_its_infinities():
    """A NaN or infinity in one channel's row stays in that channel, and in its own sequence's sums."""
    p = make(2, 30, 130, 1, 16, F32, 7)
    want, tol = reference(p)
    p["x"][0, 10, 65] = float("nan")
    p["z"][0, 3, 2] = float("inf")
    got = run(p)
    y = got["y"].cpu().double()
    fine = torch.ones_like(y, dtype=torch.bool)
    fine[0, 10:, 65] = False
    fine[0, 3, 2] = False
    assert ((y - want["y"]).abs() <= tol["y"])[fine].all() and torch.isnan(y[0, 10:, 65]).all()
    assert ((got["dB"].cpu()[1].double() - want["dB"][1]).abs() <= tol["dB"][1] + 1e-37).all()


@pytest.mark.parametrize("N", [16, 40])
def test_a_sequence_ends_with_its_infinities(N):
    """What is not finite in one packed sequence reaches neither the next one nor, backwards, the one before."""
    T = 150
    p = make(1, T, 70, 1, N, F32, 13)
    start = torch.zeros((1, T), dtype=torch.uint8)
    start[0, [40, 90]] = 1
    p["S0"], p["dS"] = None, None
    want, tol = reference(p, True, start)
    for bad in ("nan", "inf"):
        q = dict(p, x=p["x"].clone(), dy=p["dy"].clone())
        q["x"][0, 50, 69] = float(bad)
        q["dy"][0, 60, 3] = float(bad)
        got = run(q, True, start)
        for k in ("y", "dx", "ddt", "dz", "dB", "dC"):
            e = (got[k].cpu().double().reshape(want[k].shape) - want[k]).abs() <= tol[k] + 1e-37
            assert e[:, :40].all() and e[:, 90:].all(), (k, bad)
        assert ((got["S"].cpu().double() - want["S"]).abs() <= tol["S"]).all()


@pytest.mark.parametrize("name", ["x", "dt", "B", "C", "z", "dy"])
@pytest.mark.parametrize("N", [16, 40])
def test_a_sequence_ends_with_its_infinities_at_its_ends(N, name):
    """The same for its first and last token and those next to them, whichever tensor holds them."""
    T = 150
    p = make(1, T, 70, 1, N, F32, 14)
    start = torch.zeros((1, T), dtype=torch.uint8)
    start[0, [40, 90]] = 1
    want, tol = reference(p, True, start)
    for bad in ("nan", "inf", "-inf"):
        for t in (40, 41, 47, 81, 88, 89):
            q = dict(p)
            q[name] = p[name].clone()
            q[name][0, t, ..., 1] = float(bad)
            got = run(q, True, start)
            for k in ("y", "dx", "ddt", "dz", "dB", "dC"):
                e = (got[k].cpu().double().reshape(want[k].shape) - want[k]).abs() <= tol[k] + 1e-37
                assert e[:, :40].all() and e[:, 90:].all(), (k, bad, t)
            for k in ("S", "dS0"):
                assert ((got[k].cpu().double() - want[k]).abs() <= tol[k]).all(), (k, bad, t)


def test_extreme_steps():
    """Steps so large that nothing is left of a state, and so small that nothing happens."""
    p = make(1, 20, 64, 1, 16, F32, 9)
    p["dt"][0, 5] = 80.0
    p["dt"][0, 6] = -80.0
    p["dt"][0, 7] = -200.0
    p["dt_bias"] = None
    want, tol = reference(p)
    got = run(p)
    # |dt| up to 200: the exponential of its magnitude is off by 1.25 half steps of that, 250 in place of 20
    check(got, want, {k: 4 * v + 250 * 2.0 ** -24 * want[k].abs() for k, v in tol.items()})
    assert all(torch.isfinite(v).all() for v in got.values())


def test_gradients_against_differences():
    """d/ds of <dy, y> + <dS, S> along a random direction by central differences in fp32 (1e-3 and 64 of its
    half steps over the step, 2^-6: some 2.5e-4; and the third derivative)."""
    p = make(2, 20, 20, 2, 5, F32, 4)
    c = {k: v.to(DEV) for k, v in p.items()}
    got = run(p)
    g = torch.Generator().manual_seed(5)
    for name in NAMES:
        v = torch.randn(c[name].shape, generator=g).to(DEV)
        v = v * c[name].abs() if name == "A" else v
        s = 2.0 ** -6

        def loss(k):
            q = dict(c, **{name: c[name] + k * v})
            y, S = sdm.sdm_selective_scan_forward(q["x"], q["dt"], q["A"], q["B"], q["C"], q["D"], q["z"], q["dt_bias"], True, q["S0"])
            return float((y.double() * c["dy"].double()).sum() + (S.double() * c["dS"].double()).sum())

        t = got["d" + name].double().reshape(v.shape) * v.double()
        assert abs((loss(s) - loss(-s)) / (2 * s) - float(t.sum())) <= 2e-3 * float(t.abs().sum()), name


def test_far_rows():
    """Offsets beyond 2^31 elements between sequences."""
    p = make(2, 9, 64, 1, 16, BF, 4)
    far = torch.zeros((1 << 31) + 4096, dtype=BF, device=DEV)
    x = far.as_strided((2, 9, 64), ((1 << 31) + 64, 64, 1))
    x.copy_(p["x"])
    check(run(p, x=x), *reference(p))


@pytest.mark.parametrize("break_it", [
    lambda c: dict(x=c["x"].transpose(1, 2)), lambda c: dict(dt=c["dt"].float()), lambda c: dict(z=c["z"][:, :3]),
    lambda c: dict(A=c["A"].to(BF)), lambda c: dict(A=c["A"][:, :4]), lambda c: dict(Bm=c["B"][..., :4]), lambda c: dict(Cm=c["C"][:, :, 0]),
    lambda c: dict(D=c["D"][:5]), lambda c: dict(dt_bias=c["D"].double()), lambda c: dict(S0=c["S0"].to(BF)), lambda c: dict(S0=c["S0"][:1]),
    lambda c: dict(start=torch.zeros((2, 5), device=DEV)), lambda c: dict(lengths=torch.zeros(2, device=DEV)),
    lambda c: dict(x=c["x"].cpu()), lambda c: dict(workspace=torch.zeros(4, device=DEV))])
def test_refusals(break_it):
    c = {k: v.to(DEV) for k, v in make(2, 6, 64, 1, 16, BF, 0).items()}
    good = dict(x=c["x"], dt=c["dt"], A=c["A"], Bm=c["B"], Cm=c["C"], D=c["D"], z=c["z"], dt_bias=c["dt_bias"], S0=c["S0"])
    sdm.sdm_selective_scan_forward(**good)
    with pytest.raises(ValueError):
        sdm.sdm_selective_scan_forward(**dict(good, **break_it(c)))


def test_refusals_of_the_library():
    c = {k: v.to(DEV) for k, v in make(2, 6, 64, 1, 16, BF, 0).items()}
    z = lambda *s: torch.zeros(s, dtype=BF, device=DEV)  # noqa: E731
    with pytest.raises((sdm.SdmError, ValueError)):
        sdm.sdm_selective_scan_forward(c["x"], c["dt"], torch.zeros((64, 65), device=DEV), z(2, 6, 65), z(2, 6, 65))
    with pytest.raises(sdm.SdmError):
        sdm.sdm_selective_scan_forward(c["x"], c["dt"], c["A"], c["B"], c["C"], y=c["x"])
    with pytest.raises(ValueError):
        sdm.sdm_selective_scan_backward(c["dy"], c["x"], c["dt"], c["A"], c["B"], c["C"], out={"dz": c["z"]})
    with pytest.raises(sdm.SdmError):
        sdm.sdm_selective_scan_backward(c["dy"], c["x"], c["dt"], c["A"], c["B"], c["C"], out={"dx": c["dy"]})
    with pytest.raises(sdm.SdmError):
        sdm.sdm_selective_scan_backward(c["dy"], c["x"], c["dt"], c["A"], c["B"], c["C"],
                                        workspace=torch.zeros(64, dtype=torch.uint8, device=DEV))
