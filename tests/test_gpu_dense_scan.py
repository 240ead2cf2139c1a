"""The dense gated recurrence and its gradients against a token-by-token walk in
64 bits.

Tolerances: every output is a sum of products, and each product passes through
at most n roundings of fp32 (half a step each, 2^-24 relative): its own
contractions over dk and dv, a chunk's sums and decays, and a few per chunk
crossed. So an output is off by at most n 2^-24 times the same sum taken over
the magnitudes, which a second walk with all inputs' magnitudes gives. d/d ln
alpha is a running sum over at most 512 tokens of q.dq - k.dk from the segment's
end, so its magnitude is that of the whole sum.
"""
import pytest
import torch

import sparse_memory_linear_amd as sdm

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
BF, F32 = torch.bfloat16, torch.float32
EPS = torch.finfo(F32).eps / 2
SEGMENT = 512


def make(B, H, T, dk, dv, dtype, seed, gates="mid", states=True):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    x = {"q": r(B, H, T, dk).mul_(dk ** -0.5).to(dtype), "k": r(B, H, T, dk).mul_(dk ** -0.5).to(dtype),
         "v": r(B, H, T, dv).to(dtype), "alpha": torch.sigmoid(r(B, H, T) * 0.5 + 2.0),
         "beta": torch.sigmoid(r(B, H, T)), "dy": r(B, H, T, dv)}
    if gates == "extreme":  # zeros (a new sequence), ones, tiny ones, writes of nothing
        u = torch.rand((B, H, T), generator=g)
        x["alpha"] = torch.where(u < 0.05, 0.0, torch.where(u < 0.3, 1.0, torch.where(u < 0.4, 1e-30, x["alpha"])))
        x["beta"] = torch.where(torch.rand((B, H, T), generator=g) < 0.2, 0.0, x["beta"])
    x["S0"] = r(B, H, dk, dv) if states else None
    x["dS"] = r(B, H, dk, dv) if states else None
    return x


def walk(x, magnitudes=False):
    """y, S and all gradients in 64 bits, on the CPU, one token at a time."""
    f = lambda t: None if t is None else (t.double().abs() if magnitudes else t.double())  # noqa: E731
    q, k, v, al, be, dy, S0, dS = (f(x[n]) for n in ("q", "k", "v", "alpha", "beta", "dy", "S0", "dS"))
    B, H, T, dk = q.shape
    dv = v.shape[-1]
    S = torch.zeros(B, H, dk, dv, dtype=torch.float64) if S0 is None else S0
    y, states = torch.zeros(B, H, T, dv, dtype=torch.float64), [S]
    for t in range(T):
        S = al[:, :, t, None, None] * S + be[:, :, t, None, None] * k[:, :, t, :, None] * v[:, :, t, None, :]
        states.append(S)
        y[:, :, t] = (q[:, :, t, :, None] * S).sum(-2)
    o = {"y": y, "S": S, "dq": torch.zeros_like(q), "dk": torch.zeros_like(k), "dv": torch.zeros_like(v),
         "dlog_alpha": torch.zeros_like(al), "dbeta": torch.zeros_like(be)}
    G = torch.zeros_like(S) if dS is None else dS
    for t in reversed(range(T)):
        G = G + q[:, :, t, :, None] * dy[:, :, t, None, :]
        o["dq"][:, :, t] = (states[t + 1] * dy[:, :, t, None, :]).sum(-1)
        Gv = (G * v[:, :, t, None, :]).sum(-1)
        o["dk"][:, :, t] = be[:, :, t, None] * Gv
        o["dv"][:, :, t] = be[:, :, t, None] * (G * k[:, :, t, :, None]).sum(-2)
        o["dbeta"][:, :, t] = (k[:, :, t] * Gv).sum(-1)
        aS = al[:, :, t, None, None] * states[t]
        o["dlog_alpha"][:, :, t] = (G * aS).sum((-1, -2))
        G = al[:, :, t, None, None] * G
    o["dS0"] = G
    if magnitudes:  # the running sum's terms, over the tokens of up to a segment ahead, and its start
        c = (q * o["dq"]).sum(-1) + (k * o["dk"]).sum(-1)
        run = torch.nn.functional.pad(c.flip(-1).cumsum(-1).flip(-1), (0, 1))  # run[t]: tokens t and behind
        ahead = torch.arange(T).add(SEGMENT).clamp_max(T)
        E = torch.nn.functional.pad(o["dlog_alpha"], (0, 1))
        E[..., T] = 0.0 if dS is None else (dS * S).sum((-1, -2))
        # the segment's end lies at most SEGMENT tokens ahead, with a value E there
        far = torch.stack([E[..., t + 1:t + SEGMENT + 1].amax(-1) for t in range(T)], -1)
        o["dlog_alpha"] = run[..., :T] - run[..., ahead] + far
    return o


def roundings(T, dk, dv):
    chunks = (T + 31) // 32
    return 2 * (dk + dv) + 2 * 64 + 64 + 4 * chunks + 64


def check(got, want, mag, n, names):
    for name in names:
        w, m = want[name], mag[name]
        e = (got[name].cpu().double() - w).abs()
        tol = n * EPS * m + 1e-37
        assert torch.isfinite(got[name]).all(), name
        worst = (e / tol).max().item() if e.numel() else 0.0
        assert worst <= 1.0, (name, worst, e.max().item())


def dev(x):
    return {n: None if t is None else t.to(DEV) for n, t in x.items()}


def forward(x, **kw):
    y, S = sdm.sdm_dense_scan_forward(x["q"], x["k"], x["v"], x["alpha"], x["beta"], x["S0"], **kw)
    return {"y": y, "S": S}


def backward(x, **kw):
    return sdm.sdm_dense_scan_backward(x["q"], x["k"], x["v"], x["alpha"], x["beta"], x["dy"], x["S0"], x["dS"], **kw)


GRADS = ("dq", "dk", "dv", "dlog_alpha", "dbeta", "dS0")

SIZES = [  # B, H, T, dk, dv: one token to several segments, tiles filled and not
    (1, 1, 1, 8, 8), (3, 2, 1, 128, 128), (2, 2, 3, 256, 72), (1, 3, 8, 64, 40), (1, 1, 9, 16, 8),
    (2, 1, 31, 40, 24), (1, 2, 64, 64, 64), (2, 2, 65, 72, 136), (1, 2, 300, 128, 128),
    (1, 1, 517, 256, 256), (1, 1, 130, 64, 256), (1, 1, 140, 128, 200), (1, 1, 256, 64, 72), (1, 1, 257, 72, 64), (2, 1, 1100, 96, 80), (1, 2, 577, 200, 64), (1, 1, 1537, 32, 128),
]


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("B,H,T,dk,dv", SIZES)
def test_forward_and_backward(B, H, T, dk, dv, dtype):
    x = make(B, H, T, dk, dv, dtype, 7 * T + dk + dv)
    want, mag, n = walk(x), walk(x, True), roundings(T, dk, dv)
    g = dev(x)
    check(forward(g), want, mag, n, ("y", "S"))
    check(backward(g), want, mag, n, GRADS)


@pytest.mark.parametrize("B,H,T,dk,dv,dtype", [(2, 2, 5, 64, 64, BF), (1, 2, 700, 128, 64, BF), (1, 2, 700, 64, 128, F32)])
@pytest.mark.parametrize("states", [True, False], ids=["states", "zeros"])
def test_extreme_gates_and_missing_states(B, H, T, dk, dv, dtype, states):
    x = make(B, H, T, dk, dv, dtype, 5, gates="extreme", states=states)
    want, mag, n = walk(x), walk(x, True), roundings(T, dk, dv)
    g = dev(x)
    check(forward(g), want, mag, n, ("y", "S"))
    check(backward(g), want, mag, n, GRADS)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("T0,T1", [(64, 40), (70, 90), (17, 3), (600, 700), (512, 512)])
def test_a_gate_of_zero_keeps_two_sequences_apart(T0, T1, dtype):
    """The second sequence's rows are 2^10 times larger, its gradients' products 2^40 times: a
    rounding of them that passed the gate would be far beyond the first one's bound."""
    x, z = make(1, 2, T0, 64, 40, dtype, T0, states=False), make(1, 2, T1, 64, 40, dtype, T1, states=False)
    z["alpha"][:, :, 0] = 0.0
    both = {n: None if x[n] is None else torch.cat([x[n], z[n] * (1024 if n in ("q", "k", "v", "dy") else 1)], 2) for n in x}
    want, mag, n = walk(x), walk(x, True), roundings(T0 + T1, 64, 40)
    g = dev(both)
    got, y = backward(g), forward(g)["y"]
    first = {m: got[m][:, :, :T0] for m in GRADS if m != "dS0"}
    check({**first, "dS0": got["dS0"], "y": y[:, :, :T0]}, want, mag, n, ("y",) + GRADS)
    assert (got["dlog_alpha"][:, :, T0] == 0).all()


def test_state_in_place_and_preallocated_outputs():
    for T in (1, 4, 40, 1500):
        g = dev(make(2, 2, T, 64, 96, BF, T))
        want = forward(g)
        big = torch.full((2 * 2 * T * 96 + 64,), 7.0, device=DEV)
        y = big[32:-32].view(2, 2, T, 96)
        S = g["S0"].clone()
        y2, S2 = sdm.sdm_dense_scan_forward(g["q"], g["k"], g["v"], g["alpha"], g["beta"], S, S, y)
        assert y2.data_ptr() == y.data_ptr() and S2.data_ptr() == S.data_ptr()
        assert torch.equal(y, want["y"]) and torch.equal(S, want["S"])
        assert (big[:32] == 7).all() and (big[-32:] == 7).all()  # nothing before or behind is touched
        dS = g["dS"].clone()
        ref = backward(g)
        g["dS"] = dS
        got = backward(g, out={"dS0": dS})
        assert got["dS0"].data_ptr() == dS.data_ptr()
        for name in GRADS:
            assert torch.equal(got[name], ref[name]), name


def test_no_tokens_pass_the_states_on():
    x = dev(make(2, 3, 4, 16, 8, F32, 1))
    z = {n: x[n][:, :, :0].contiguous() for n in ("q", "k", "v", "alpha", "beta", "dy")}
    z["S0"], z["dS"] = x["S0"], x["dS"]
    got = forward(z)
    assert got["y"].shape == (2, 3, 0, 8) and torch.equal(got["S"], x["S0"])
    assert torch.equal(backward(z)["dS0"], x["dS"])
    z["S0"] = None
    assert (forward(z)["S"] == 0).all()


def test_states_that_are_not_wanted():
    """Through the C ABI: no last state, and no gradient of the first."""
    from sparse_memory_linear_amd import binding
    lib, p = binding.lib(), lambda t: t.data_ptr()  # noqa: E731
    for T in (1, 40, 1500):
        g = dev(make(2, 2, T, 64, 96, BF, T))
        want, grads = forward(g), backward(g)
        ws = torch.empty(max(16, sdm.sdm_dense_scan_workspace_bytes(2, 2, T, 64, 96)), dtype=torch.uint8, device=DEV)
        y = torch.empty_like(want["y"])
        st = torch.cuda.current_stream().cuda_stream
        args = [p(g[m]) for m in ("q", "k", "v")] + [1, p(g["alpha"]), p(g["beta"])]
        assert lib.sdm_dense_scan_forward(*args, p(g["S0"]), None, p(y), 2, 2, T, 64, 96, p(ws), ws.numel(), st) == 0
        ws = torch.empty(sdm.sdm_dense_scan_backward_workspace_bytes(2, 2, T, 64, 96), dtype=torch.uint8, device=DEV)
        out = {m: torch.empty_like(grads[m]) for m in GRADS[:-1]}
        assert lib.sdm_dense_scan_backward(*args, p(g["dy"]), p(g["S0"]), p(g["dS"]), *(p(out[m]) for m in GRADS[:-1]), None,
                                           2, 2, T, 64, 96, p(ws), ws.numel(), st) == 0
        torch.cuda.synchronize()
        assert torch.equal(y, want["y"])
        for m in out:
            assert torch.equal(out[m], grads[m]), m


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_split_calls_continue_the_sequence(dtype):
    x = make(1, 2, 900, 64, 64, dtype, 3)
    want, mag, n = walk(x), walk(x, True), roundings(900, 64, 64) + 128
    g = dev(x)
    at = [0, 1, 2, 70, 611, 900]
    S, ys, starts = g["S0"], [], []
    cut = lambda a, b: {m: g[m][:, :, a:b].contiguous() for m in ("q", "k", "v", "alpha", "beta", "dy")}  # noqa: E731
    for a, b in zip(at, at[1:]):
        c = cut(a, b)
        starts.append(S)
        y, S = sdm.sdm_dense_scan_forward(c["q"], c["k"], c["v"], c["alpha"], c["beta"], S)
        ys.append(y)
    check({"y": torch.cat(ys, 2), "S": S}, want, mag, n, ("y", "S"))
    parts, dS = [], g["dS"]
    for (a, b), S in reversed(list(zip(zip(at, at[1:]), starts))):
        c = cut(a, b)
        parts.insert(0, sdm.sdm_dense_scan_backward(c["q"], c["k"], c["v"], c["alpha"], c["beta"], c["dy"], S, dS))
        dS = parts[0]["dS0"]
    got = {m: torch.cat([p[m] for p in parts], 2) for m in GRADS[:-1]}
    got["dS0"] = dS
    check(got, want, mag, n, GRADS)


def test_gradients_against_differences():
    """The directional derivative of the loss, by differences of the walk in 64
    bits. A step of 2^-20 leaves an error of the third derivative's size, 2^-40, and
    2^-53 / 2^-20 of rounding: both far below the kernels' own."""
    x = make(1, 2, 90, 24, 16, F32, 11)
    g = backward(dev(x))
    gen = torch.Generator().manual_seed(2)
    loss = lambda z: sum((walk(z)[a] * z0).sum() for a, z0 in (("y", x["dy"].double()), ("S", x["dS"].double())))  # noqa: E731
    names = {"q": "dq", "k": "dk", "v": "dv", "beta": "dbeta", "S0": "dS0", "alpha": "dlog_alpha"}
    for a, b in names.items():
        d = torch.randn(x[a].shape, generator=gen, dtype=torch.float64)
        sides = []
        for s in (2.0 ** -20, -2.0 ** -20):
            z = {m: t.double() for m, t in x.items()}
            z[a] = z[a] * torch.exp(s * d) if a == "alpha" else z[a] + s * d
            sides.append(loss(z))
        want = (sides[0] - sides[1]) / 2.0 ** -19
        got = (g[b].cpu().double() * d).sum()
        size = (g[b].cpu().double() * d).abs().sum()
        assert abs(want - got) <= 1e-5 * size, (a, float(want), float(got))


def test_captured_and_replayed_between_other_work():
    for T in (2, 130, 1300):
        g = dev(make(2, 2, T, 64, 64, BF, T))
        want_f, want_b = forward(g), backward(g)
        outs = {}
        torch.cuda.synchronize()
        s = torch.cuda.Stream()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.stream(s):
            forward(g), backward(g)
            torch.cuda.synchronize()
            with torch.cuda.graph(graph, stream=s):
                outs.update(forward(g))
                outs.update(backward(g))
        for _ in range(4):
            for t in outs.values():
                t.fill_(float("nan"))
            other = dev(make(1, 2, 70, 64, 64, BF, 1))
            forward(other)
            graph.replay()
            backward(other)
            torch.cuda.synchronize()
            for name, t in outs.items():
                assert torch.equal(t, want_f[name] if name in want_f else want_b[name]), name


def test_two_streams_at_once():
    a, b = dev(make(2, 2, 1200, 128, 64, BF, 1)), dev(make(1, 3, 800, 64, 128, F32, 2))
    want = [forward(a), backward(a), forward(b), backward(b)]
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(3):
        with torch.cuda.stream(s1):
            r1 = [forward(a), backward(a)]
        with torch.cuda.stream(s2):
            r2 = [forward(b), backward(b)]
        torch.cuda.synchronize()
        for got, ref in zip(r1 + r2, want):
            for name in ref:
                assert torch.equal(got[name], ref[name]), name


def test_offsets_beyond_32_bits():
    """One stream of 8.6 M tokens, 256 wide: rows lie beyond 2^32 bytes. A gate of 0
    near the end starts the sequence anew, so the tokens behind it equal a call of their own."""
    T, n, d = 8_600_001, 200, 256
    gen = torch.Generator(device=DEV).manual_seed(0)
    x = {m: torch.empty((1, 1, T, d), dtype=BF, device=DEV).normal_(generator=gen) for m in ("q", "k", "v")}
    al = torch.full((1, 1, T), 0.9, device=DEV)
    al[..., T - n] = 0.0
    be = torch.rand((1, 1, T), generator=gen, device=DEV)
    y, S = sdm.sdm_dense_scan_forward(x["q"], x["k"], x["v"], al, be)
    end = {m: t[:, :, T - n:].clone() for m, t in x.items()}
    y2, S2 = sdm.sdm_dense_scan_forward(end["q"], end["k"], end["v"], al[..., T - n:].clone(), be[..., T - n:].clone())
    # the same sums in other chunks: n roundings of the magnitudes, here of 256 + 10 (decay 0.9) products
    assert (y[:, :, T - n:] - y2).abs().max() <= 1e-5 * y2.abs().max()
    assert (S - S2).abs().max() <= 1e-5 * S2.abs().max()


def test_backward_offsets_beyond_32_bits():
    """4.3 M tokens of 256 fp32 gradients a row: as above, the tokens behind a gate of 0 have the
    gradients of a call of their own (but for that gate's, which is 0)."""
    T, n, d = 4_300_001, 150, 256
    gen = torch.Generator(device=DEV).manual_seed(1)
    x = {m: torch.empty((1, 1, T, d), dtype=BF, device=DEV).normal_(generator=gen) for m in ("q", "k", "v")}
    x["dy"] = torch.empty((1, 1, T, d), device=DEV).normal_(generator=gen)
    x["alpha"] = torch.full((1, 1, T), 0.9, device=DEV)
    x["alpha"][..., T - n] = 0.0
    x["beta"] = torch.rand((1, 1, T), generator=gen, device=DEV)
    x["S0"] = x["dS"] = None
    whole = backward(x)
    end = {m: None if t is None else t[:, :, T - n:].clone() for m, t in x.items()}
    part = backward(end)
    for name in GRADS[:-1]:
        a, b = whole[name][:, :, T - n:], part[name]
        assert (a - b).abs().max() <= 1e-5 * b.abs().max(), name  # the same sums in other chunks
    assert (whole["dlog_alpha"][..., T - n] == 0).all()


def test_refusals():
    g = dev(make(1, 2, 9, 16, 8, BF, 1))
    args = [g[m] for m in ("q", "k", "v", "alpha", "beta")]
    bad = lambda i, t: [t if j == i else a for j, a in enumerate(args)]  # noqa: E731
    for a in (bad(1, g["k"].float()), bad(2, g["v"][:, :1]), bad(3, g["alpha"].double()),
              bad(0, g["q"].transpose(2, 3).contiguous().transpose(2, 3)), bad(4, g["beta"].cpu())):
        with pytest.raises(ValueError):
            sdm.sdm_dense_scan_forward(*a)
    with pytest.raises(ValueError):
        sdm.sdm_dense_scan_forward(*args, g["S0"].to(BF))
    with pytest.raises(ValueError):
        sdm.sdm_dense_scan_backward(*args, g["dy"].to(BF))
    q = torch.zeros((1, 2, 9, 264), dtype=BF, device=DEV)
    with pytest.raises((ValueError, sdm.SdmError)):
        sdm.sdm_dense_scan_forward(q, q, g["v"], g["alpha"], g["beta"])
    long = dev(make(1, 2, 2000, 16, 8, BF, 1))
    with pytest.raises(sdm.SdmError):
        forward(long, workspace=torch.empty(64, dtype=torch.uint8, device=DEV))


def test_values_of_other_ranks_are_refused():
    g = dev(make(1, 2, 9, 16, 8, BF, 1))
    for v in (g["v"][..., 0].contiguous(), g["v"][..., None].contiguous()):
        with pytest.raises(ValueError):
            sdm.sdm_dense_scan_forward(g["q"], g["k"], v, g["alpha"], g["beta"])
        with pytest.raises(ValueError):
            sdm.sdm_dense_scan_backward(g["q"], g["k"], v, g["alpha"], g["beta"], g["dy"])


def test_single_products_keep_all_of_fp32():
    """y = q S0 with one factor a row (gates of 1, writes of nothing) is one fp32 x fp32 product of
    operand planes. The matrix instructions round a sum to one of its two neighbours, not always the
    nearer one (products of two planes by three, where nothing is left out, are up to 1.93 half steps
    off, to either side): less than 2 half steps for the last sum, 2 * 2^-8 for each of the two before
    it, 2^-15 for the others. The plane products left out are 2^-24 of the product at most (a middle
    plane is at most 2^-8 of its value and a low one 2^-17: 2 * 2^-25 + 2^-34), 1 half step. So 3.1
    bounds them all; and of either sign each, they are nothing on average (the mean over 2^17 values
    with a deviation of 0.6 is within 0.01; 0.1 bounds it)."""
    n, d = 32, 64
    g = torch.Generator().manual_seed(3)
    a, S0 = torch.randn((n, 1, d), generator=g), torch.randn((n, 1, d, d), generator=g)
    q = torch.diag_embed(a)
    one, zero = torch.ones(n, 1, d), torch.zeros(n, 1, d)
    rows = torch.randn((n, 1, d, d), generator=g)
    y, _ = sdm.sdm_dense_scan_forward(q.to(DEV), rows.to(DEV), rows.to(DEV), one.to(DEV), zero.to(DEV), S0.to(DEV))
    want = a.double()[..., None] * S0.double()
    off = (y.cpu().double() - want) / want / EPS
    assert off.abs().max() <= 3.1, off.abs().max().item()
    assert off.mean().abs() <= 0.1, off.mean().item()


# Segments of 512 tokens (16 chunks; many streams) and errors in the mean.
CHUNK = 32


def magnitudes(x):
    return walk({m: None if t is None else t.double().abs() for m, t in x.items()})


def dot_magnitudes(x, o, mag):
    """dlog_alpha's terms, in magnitude: its sums begin anew every CHUNK tokens. Up to its chunk's end a token
    adds q.dq and k.dk; E at a chunk's end is that at the segment's end (a product of the two states) and, per
    chunk between, what crosses its bounds: never more than E's own terms there, each taken three times at
    most (from its product or the chunk behind, the chunk before, and the sum)."""
    B, H, T = x["alpha"].shape
    E = torch.nn.functional.pad(o["dlog_alpha"], (0, 1))
    if x["dS"] is not None:
        E[..., T] = (x["dS"].double().abs() * o["S"]).sum((-1, -2)) if mag else (x["dS"].double() * o["S"]).sum((-1, -2))
    a = lambda t: t.double().abs() if mag else t.double()  # noqa: E731
    terms = [(a(x[m]) * o["d" + m]).sum(-1) for m in ("q", "k")]
    f, g = (lambda z: z, lambda z: z) if mag else (torch.square, torch.sqrt)
    out = torch.zeros_like(o["dlog_alpha"])
    for t0 in range(0, T, CHUNK):
        t1, last = min(T, t0 + CHUNK), min(T, (t0 // SEGMENT + 1) * SEGMENT)
        for c in terms:
            out[:, :, t0:t1] += f(c[:, :, t0:t1]).flip(-1).cumsum(-1).flip(-1)
        for b in {*range(t1, last, CHUNK), last}:
            out[:, :, t0:t1] += 3 * f(E[:, :, b, None])
    return g(out)


def in_the_mean(got, want, x, T, dk, dv):
    """Errors against the outputs in the mean square. A sum's roundings are of either sign, and its partial
    sums no larger than the result in the mean, so m of them leave sqrt(m) times one: at most 2 half steps
    over sqrt(3) where a matrix instruction rounds to either neighbour. m: 6 plane products per 32 of a width
    for each of two contractions, 7 per chunk that the state crosses, 30 for decays, products and sums. A
    plane that is lost is 2^-17 of its operand: some 30 half steps in the mean of its products."""
    m = 12 * ((max(dk, dv) + 31) // 32) + 7 * ((T + CHUNK - 1) // CHUNK) + 30
    rms = lambda t: t.square().mean().sqrt().item()  # noqa: E731
    for name in ("y", "S") + GRADS:
        size = rms(dot_magnitudes(x, want, False) if name == "dlog_alpha" else want[name])
        e = rms(got[name].cpu().double() - want[name])
        assert e <= (4 * m / 3) ** 0.5 * EPS * size, (name, e / size / EPS, (4 * m / 3) ** 0.5)


def check_streams(x, streams, mean=True):
    """All streams in one call, some of them against the walk."""
    g = dev(x)
    got = {**forward(g), **backward(g)}
    pick = lambda z: {m: None if t is None else t.flatten(0, 1)[streams][:, None] for m, t in z.items()}  # noqa: E731
    x, got = pick(x), pick(got)
    (T, dk), dv = x["q"].shape[2:], x["v"].shape[3]
    want, mag = walk(x), magnitudes(x)
    mag["dlog_alpha"] = dot_magnitudes(x, mag, True)
    check(got, want, mag, roundings(T, dk, dv), ("y", "S") + GRADS)
    if mean:
        in_the_mean(got, want, x, T, dk, dv)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("B,H,T,dk,dv", [(1, 2, 300, 128, 128), (2, 1, 130, 256, 256), (1, 1, 577, 200, 64), (2, 2, 96, 64, 40)])
def test_errors_in_the_mean(B, H, T, dk, dv, dtype):
    check_streams(make(B, H, T, dk, dv, dtype, T + dv), list(range(B * H)))


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("gates", ["mid", "extreme", "near one"])
@pytest.mark.parametrize("B,H,T,dk,dv,streams", [(64, 8, 1100, 8, 16, [0, 7, 300, 511]), (8, 32, 1100, 72, 136, [3, 255]),
                                                 (8, 8, 2085, 128, 128, [63])])
def test_segments_of_many_chunks(B, H, T, dk, dv, streams, gates, dtype):
    """With 512 streams and column slabs a segment takes 512 tokens, with 64 streams of 2085 tokens 288 (the last one fewer)."""
    x = make(B, H, T, dk, dv, dtype, T + dk, gates="extreme" if gates == "extreme" else "mid")
    if gates == "near one":
        x["alpha"] = 1 - (1 - x["alpha"]) / 64
    check_streams(x, streams, gates != "extreme")


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_roundings_of_a_large_token_stay_in_its_chunk(dtype):
    """Token 400 has rows 2^10 times the others', products 2^40 times; around it gates of 1/2 let nothing
    of that reach beyond a chunk or two. A sum over the whole segment would carry roundings of 2^16 on."""
    x = make(64, 8, 1030, 16, 8, dtype, 4)
    x["alpha"][:, :, 300:430] = 0.5
    for m in ("q", "k", "v", "dy"):
        x[m][:, :, 400] *= 1024
    check_streams(x, [0, 200, 511], False)
