"""The operators of a selective state-space layer in use together, and beside the others: norm, projections,
convolution, scan, projection, forwards and backwards; a dense gated layer whose q, k and v come through the convolution;
decoding; streams and graphs.

Tolerance: each operator's result is off by at most some 600 roundings of 2^-24 times its terms' magnitudes, 4e-5; a
gradient passes through eight of them, so 3e-4 of the largest magnitude bounds what they add up to.
"""
import pytest
import torch

import sparse_memory_linear_amd as sdm
from sparse_memory_linear_amd import binding

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
EPS, TOL = 1e-5, 3e-4
PARAMS = ("x", "gamma", "bias", "Win", "cw", "cb", "Wx", "Wdt", "dt_bias", "A", "D", "Wo")


def layer(B=2, T=130, d=48, inner=96, N=12, R=6, K=4, seed=0):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    return {"x": r(B, T, d), "res": r(B, T, d), "gamma": 1 + 0.1 * r(d), "bias": 0.1 * r(d), "Win": r(d, 2 * inner) / d ** 0.5,
            "cw": r(inner, K) / K ** 0.5, "cb": 0.1 * r(inner), "Wx": r(inner, R + 2 * N) / inner ** 0.5, "Wdt": r(R, inner) / R ** 0.5,
            "dt_bias": r(inner) - 2, "A": -torch.exp(0.3 * r(inner, N)), "D": r(inner), "Wo": r(inner, d) / inner ** 0.5, "c": r(B, T, d)}


def reference(p):
    """The layer in 64 bits by torch's own derivatives; loss <c, out>."""
    p = {k: v.double().requires_grad_() for k, v in p.items()}
    (B, T, d), (inner, K), N = p["x"].shape, p["cw"].shape, p["A"].shape[1]
    h = p["x"] + p["res"]
    n = torch.nn.functional.layer_norm(h, (d,), p["gamma"], p["bias"], EPS)
    u, z = (n @ p["Win"]).split(inner, -1)
    padded = torch.nn.functional.pad(u, (0, 0, K - 1, 0))
    u = torch.nn.functional.silu(sum(padded[:, j:j + T] * p["cw"][:, j] for j in range(K)) + p["cb"])
    low, Bm, Cm = (u @ p["Wx"]).split([p["Wdt"].shape[0], N, N], -1)
    delta = torch.nn.functional.softplus(low @ p["Wdt"] + p["dt_bias"])
    S, ys = torch.zeros(B, inner, N, dtype=torch.float64), []
    for t in range(T):
        S = (delta[:, t, :, None] * p["A"]).exp() * S + (delta[:, t] * u[:, t])[..., None] * Bm[:, t, None]
        ys.append((S * Cm[:, t, None]).sum(-1))
    y = (torch.stack(ys, 1) + p["D"] * u) * torch.nn.functional.silu(z)
    out = y @ p["Wo"] + h
    grads = torch.autograd.grad((out * p["c"]).sum(), [p[k] for k in PARAMS])
    return out.detach(), dict(zip(PARAMS, grads))


def forward(p, conv=None, scan=None, inplace=False):
    """The layer through the library, dense products by torch; ``conv`` and ``scan`` are its states."""
    inner, N, R = p["cw"].shape[0], p["A"].shape[1], p["Wdt"].shape[0]
    a = sdm.sdm_residual_layer_norm(p["x"], p["gamma"], p["bias"], p["res"], EPS, "f32")
    xz = a["y"] @ p["Win"]
    u, conv = sdm.sdm_causal_conv_forward(xz[..., :inner], p["cw"], p["cb"], "silu", conv, conv if inplace else None)
    low = u @ p["Wx"]
    dt = low[..., :R] @ p["Wdt"]
    y, scan = sdm.sdm_selective_scan_forward(u, dt, p["A"], low[..., R:R + N], low[..., R + N:], p["D"], xz[..., inner:], p["dt_bias"], True,
                                             scan, scan if inplace else None)
    return y @ p["Wo"] + a["h"], conv, scan, (a, xz, u, low, dt, y)


def backward(p, kept):
    a, xz, u, low, dt, y = kept
    inner, N, R = p["cw"].shape[0], p["A"].shape[1], p["Wdt"].shape[0]
    flat = lambda t: t.reshape(-1, t.shape[-1])  # noqa: E731
    dxz = torch.empty_like(xz)  # the projection's gradient: the convolution writes its half in place
    s = sdm.sdm_selective_scan_backward(p["c"] @ p["Wo"].t(), u, dt, p["A"], low[..., R:R + N], low[..., R + N:], p["D"], xz[..., inner:],
                                        p["dt_bias"])
    dlow = torch.cat([s["ddt"] @ p["Wdt"].t(), s["dB"], s["dC"]], -1)
    du = s["dx"] + dlow @ p["Wx"].t()
    cv = sdm.sdm_causal_conv_backward(du, xz[..., :inner], p["cw"], p["cb"], "silu", out={"dx": dxz[..., :inner]})
    dxz[..., inner:] = s["dz"]
    n = sdm.sdm_residual_layer_norm_backward(dxz @ p["Win"].t(), a["h"], p["gamma"], p["c"], EPS)
    return {"x": n["dx"], "gamma": n["dgamma"], "bias": n["dbias"], "Win": flat(a["y"]).t() @ flat(dxz), "cw": cv["dw"], "cb": cv["dbias"],
            "Wx": flat(u).t() @ flat(dlow), "Wdt": flat(low[..., :R]).t() @ flat(s["ddt"]), "dt_bias": s["ddt_bias"], "A": s["dA"],
            "D": s["dD"], "Wo": flat(y).t() @ flat(p["c"])}


def test_layer_and_its_gradients():
    p = layer()
    want, grads = reference(p)
    c = {k: v.to(DEV) for k, v in p.items()}
    out, _, _, kept = forward(c)
    assert (out.cpu().double() - want).abs().max() <= TOL * want.abs().max()
    got = backward(c, kept)
    for k, w in grads.items():
        assert (got[k].cpu().double() - w).abs().max() <= TOL * w.abs().max(), k


def test_decoding_continues_a_prompt():
    c = {k: v.to(DEV) for k, v in layer(T=90).items()}
    whole, conv_end, scan_end, _ = forward(c)
    cut = lambda a, b: dict(c, x=c["x"][:, a:b].contiguous(), res=c["res"][:, a:b].contiguous())  # noqa: E731
    out, conv, scan, _ = forward(cut(0, 80))
    outs = [out]
    for t in range(80, 90):
        out, conv, scan, _ = forward(cut(t, t + 1), conv, scan, inplace=True)
        outs.append(out)
    assert (torch.cat(outs, 1) - whole).abs().max() <= TOL * whole.abs().max()
    assert (scan - scan_end).abs().max() <= TOL * scan_end.abs().max()
    assert (conv - conv_end).abs().max() <= TOL * conv_end.abs().max()


def dense_with_conv(c, H):
    """A dense gated layer whose q, k and v pass a convolution: heads out of one projection, no copies."""
    B, T, _ = c["x"].shape
    heads = lambda t: t.view(B, T, H, -1).transpose(1, 2)  # noqa: E731
    q, k, v = (sdm.sdm_causal_conv_forward(heads(c["x"] @ c[w]), c["w" + w[1]])[0] for w in ("Wq", "Wk", "Wv"))
    al, be = sdm.sdm_gates(c["x"], c["Wa"], c["Wb"], c["bdt"], c["A"])
    y, S = sdm.sdm_dense_scan_forward(q, k, v, al, be)
    return q, k, v, al, be, y, S


def test_dense_layer_behind_a_convolution():
    B, T, d, H, n, K = 2, 70, 32, 2, 16, 4
    g = torch.Generator().manual_seed(1)
    r = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    p = {"x": r(B, T, d), **{w: r(d, H * n) / d ** 0.5 for w in ("Wq", "Wk", "Wv")}, **{w: r(H, n, K) / 2 for w in ("wq", "wk", "wv")},
         "Wa": r(H, d) / d ** 0.5, "Wb": r(H, d) / d ** 0.5, "bdt": r(H) - 2, "A": torch.exp(0.1 * r(H))}
    c = {k: v.to(DEV) for k, v in p.items()}
    y = dense_with_conv(c, H)[5]
    f = {k: v.double() for k, v in p.items()}

    def through(w):
        x = (f["x"] @ f["W" + w]).view(B, T, H, n).transpose(1, 2)
        x = torch.nn.functional.pad(x, (0, 0, K - 1, 0))
        return torch.nn.functional.silu(sum(x[:, :, j:j + T] * f["w" + w][:, None, :, j] for j in range(K)))

    q, k, v = through("q"), through("k"), through("v")
    al = torch.exp(-f["A"][None, :, None] * torch.nn.functional.softplus((f["x"] @ f["Wa"].t()).transpose(1, 2) + f["bdt"][None, :, None]))
    be = torch.sigmoid((f["x"] @ f["Wb"].t()).transpose(1, 2))
    S, ys = torch.zeros(B, H, n, n, dtype=torch.float64), []
    for t in range(T):
        S = al[:, :, t, None, None] * S + be[:, :, t, None, None] * k[:, :, t, :, None] * v[:, :, t, None, :]
        ys.append((q[:, :, t, :, None] * S).sum(-2))
    want = torch.stack(ys, 2)
    assert (y.cpu().double() - want).abs().max() <= TOL * want.abs().max()


def step(c):
    out, conv, scan, kept = forward(c)
    return {"out": out, "conv": conv, "scan": scan, **backward(c, kept)}


def test_on_streams():
    """Two streams at once, twice over: the same bits as alone (the matrix products of torch among them)."""
    ps = [{k: v.to(DEV) for k, v in layer(seed=s, T=200).items()} for s in (0, 1)]
    want = [step(p) for p in ps]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(2):
        got = []
        for p, s in zip(ps, streams):
            with torch.cuda.stream(s):
                got.append(step(p))
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            for k in b:
                assert torch.equal(a[k], b[k]), k


def lib_step(c, out, ws):
    """The library's own calls of a layer, into tensors that exist (nothing is allocated)."""
    sdm.sdm_residual_layer_norm(c["x"], c["gamma"], c["bias"], c["res"], EPS, "f32", out={"y": out["n"], "h": out["h"]})
    sdm.sdm_causal_conv_forward(c["xz"][..., :96], c["cw"], c["cb"], "silu", None, out["conv"], y=out["u"])
    sdm.sdm_selective_scan_forward(out["u"], c["dt"], c["A"], c["Bm"], c["Cm"], c["D"], c["xz"][..., 96:], c["dt_bias"], True, None,
                                   out["S"], y=out["y"], workspace=ws)
    sdm.sdm_selective_scan_backward(c["dy"], out["u"], c["dt"], c["A"], c["Bm"], c["Cm"], c["D"], c["xz"][..., 96:], c["dt_bias"], out=out["g"],
                                    workspace=ws)
    sdm.sdm_causal_conv_backward(out["g"]["dx"], c["xz"][..., :96], c["cw"], c["cb"], "silu", out=out["cg"], workspace=ws)
    sdm.sdm_residual_layer_norm_backward(c["c"], out["h"], c["gamma"], None, EPS, out=out["ng"], workspace=ws)


def test_captured_and_replayed():
    """Two graphs that share one workspace, replayed in turn with new inputs and eager work between: every replay has the
    eager call's bits."""
    B, T, N = 2, 150, 12
    p = {k: v.to(DEV) for k, v in layer(B, T).items()}
    g = torch.Generator().manual_seed(3)
    r = lambda *s: torch.randn(s, generator=g).to(DEV)  # noqa: E731
    need = max(sdm.sdm_selective_scan_backward_workspace_bytes(B, T, 96, 1, N), sdm.sdm_selective_scan_workspace_bytes(B, T, 96, 1, N),
               sdm.sdm_causal_conv_backward_workspace_bytes(B, 1, T, 96, 4), 1 << 20)
    ws = torch.empty(need, dtype=torch.uint8, device=DEV)

    def outputs():
        e = lambda *s: torch.full(s, float("nan"), device=DEV)  # noqa: E731
        return {"n": e(B, T, 48), "h": e(B, T, 48), "conv": e(B, 3, 96), "u": e(B, T, 96), "S": e(B, 96, N), "y": e(B, T, 96),
                "g": {"dx": e(B, T, 96), "ddt": e(B, T, 96), "dz": e(B, T, 96), "dA": e(96, N), "dB": e(B, T, N), "dC": e(B, T, N),
                      "dD": e(96), "ddt_bias": e(96), "dS0": e(B, 96, N)},
                "cg": {"dx": e(B, T, 96), "dw": e(96, 4), "dbias": e(96), "dS0": e(B, 3, 96)},
                "ng": {"dx": e(B, T, 48), "dgamma": e(48), "dbias": e(48)}}

    def flat(o, at=""):
        return {f"{at}{k}{n}": t for k, v in o.items() for n, t in (flat(v, k + ".").items() if isinstance(v, dict) else [("", v)])}

    sets = []
    for _ in range(2):
        c = dict(p, xz=r(B, T, 192), dt=r(B, T, 96), Bm=r(B, T, N), Cm=r(B, T, N), dy=r(B, T, 96))
        sets.append((c, outputs()))
        lib_step(*sets[-1], ws)
    torch.cuda.synchronize()
    graphs = []
    for c, o in sets:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            lib_step(c, o, ws)
    for turn in range(4):
        for (c, o), gr in zip(sets, graphs):
            for k in ("x", "xz", "dt", "Bm", "Cm", "dy"):
                c[k].copy_(r(*c[k].shape))
            for t in flat(o).values():
                t.fill_(float("nan"))
        for gr in graphs:
            gr.replay()
        eager = []
        for c, o in sets:  # eager work between the replays, with the same workspace
            e = outputs()
            lib_step(c, e, ws)
            eager.append(e)
        torch.cuda.synchronize()
        for (c, o), e in zip(sets, eager):
            for k, t in flat(o).items():
                assert torch.equal(t, flat(e)[k]), (turn, k)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_the_library_without_strides_and_wanted_outputs(dtype):
    """The C entry points with no strides (contiguous tensors) and no optional outputs: the binding's bits, twice."""
    L, code = binding.lib(), 1 if dtype == torch.bfloat16 else 0
    B, T, D, G, N, K = 2, 77, 72, 2, 20, 4
    g = torch.Generator().manual_seed(3)
    r = lambda *s: torch.randn(s, generator=g).to(DEV)  # noqa: E731
    x, dt, dy = r(B, T, D).to(dtype), r(B, T, D).to(dtype), r(B, T, D).to(dtype)
    w, A, Bm, Cm = r(D, K), -r(D, N).abs(), r(B, T, G, N).to(dtype), r(B, T, G, N).to(dtype)
    st = torch.cuda.current_stream().cuda_stream
    p = lambda t: t.data_ptr()  # noqa: E731
    ws = lambda n: torch.empty(max(n, 16), dtype=torch.uint8, device=DEV)  # noqa: E731

    want, _ = sdm.sdm_causal_conv_forward(x, w, None, None)
    grads = sdm.sdm_causal_conv_backward(dy, x, w, None, None)
    bytes_ = L.sdm_causal_conv_backward_workspace_bytes(B, 1, T, D, K)
    for _ in range(2):
        y, dx, dw, tmp = torch.empty_like(x), torch.empty_like(x), torch.empty_like(w), ws(bytes_)
        assert L.sdm_causal_conv_forward(p(x), code, None, p(w), None, 0, None, None, None, None, p(y), B, 1, T, D, K, st) == 0
        assert L.sdm_causal_conv_backward(p(dy), p(x), code, None, p(w), None, 0, None, None, None, None, p(dx), None, p(dw),
                                          None, None, B, 1, T, D, K, p(tmp), tmp.numel(), st) == 0
        assert torch.equal(y, want) and torch.equal(dx, grads["dx"]) and torch.equal(dw, grads["dw"])

    want, _ = sdm.sdm_selective_scan_forward(x, dt, A, Bm, Cm)
    grads = sdm.sdm_selective_scan_backward(dy, x, dt, A, Bm, Cm)
    bytes_ = L.sdm_selective_scan_workspace_bytes(B, T, D, G, N), L.sdm_selective_scan_backward_workspace_bytes(B, T, D, G, N)
    for _ in range(2):
        y, dx, ddt, dA = torch.empty_like(x), torch.empty_like(x), torch.empty_like(x), torch.empty_like(A)
        dB, dC = torch.empty(Bm.shape, device=DEV), torch.empty(Bm.shape, device=DEV)
        tmp, tmp2 = ws(bytes_[0]), ws(bytes_[1])
        assert L.sdm_selective_scan_forward(p(x), p(dt), None, p(Bm), p(Cm), code, None, p(A), None, None, 1, None, None, None,
                                            None, p(y), B, T, D, G, N, p(tmp), tmp.numel(), st) == 0
        assert L.sdm_selective_scan_backward(p(dy), p(x), p(dt), None, p(Bm), p(Cm), code, None, p(A), None, None, 1, None, None,
                                             None, None, p(dx), p(ddt), None, p(dA), p(dB), p(dC), None, None, None, B, T, D, G, N,
                                             p(tmp2), tmp2.numel(), st) == 0
        for got, name in ((y, None), (dx, "dx"), (ddt, "ddt"), (dA, "dA"), (dB, "dB"), (dC, "dC")):
            assert torch.equal(got, want if name is None else grads[name]), name


def test_inputs_that_share_their_rows():
    """Inputs of stride 0 over the sequences or heads are what their copies are."""
    g = torch.Generator().manual_seed(4)
    r = lambda *s: torch.randn(s, generator=g).to(DEV)  # noqa: E731
    x, dt, w, A, Bc = r(1, 50, 40), r(1, 50, 40), r(40, 3), -r(40, 8).abs(), r(1, 50, 1, 8)
    xe, dte, Be = x.expand(3, 50, 40), dt.expand(3, 50, 40), Bc.expand(3, 50, 2, 8)
    c = lambda t: t.contiguous()  # noqa: E731
    dy = r(3, 50, 40)
    for a, b in zip(sdm.sdm_causal_conv_forward(xe, w), sdm.sdm_causal_conv_forward(c(xe), w)):
        assert torch.equal(a, b)
    a, b = sdm.sdm_causal_conv_backward(dy, xe, w, out={"dx": torch.empty_like(dy)}), sdm.sdm_causal_conv_backward(dy, c(xe), w)
    assert all(torch.equal(a[k], b[k]) for k in b)
    for a, b in zip(sdm.sdm_selective_scan_forward(xe, dte, A, Be, Be), sdm.sdm_selective_scan_forward(c(xe), c(dte), A, c(Be), c(Be))):
        assert torch.equal(a, b)
    a, b = sdm.sdm_selective_scan_backward(dy, xe, dte, A, Be, Be), sdm.sdm_selective_scan_backward(dy, c(xe), c(dte), A, c(Be), c(Be))
    assert all(torch.equal(a[k], b[k]) for k in b)
    a, b = (sdm.sdm_causal_conv_backward(dy, t, w)["dx"] for t in (xe, c(xe)))  # (its gradient does not share them)
    assert torch.equal(a, b)
