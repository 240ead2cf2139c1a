"""The operators around the sparse memory in use together: a dense layer (norm, gates, dense
recurrence) in front of a sparse one (norm, addressing with its balance loss, sparse scan),
forwards and backwards.

Tolerance: each operator's result is off by at most some 600 roundings of 2^-24 times its
terms' magnitudes, 4e-5; a gradient passes through eight of them, so 3e-4 of the largest
magnitude bounds what they add up to.
"""
import pytest
import torch

import sparse_memory_linear_amd as sdm
from sparse_memory_linear_amd import inputs

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
EPS, TOL = 1e-6, 3e-4


def layer(B=2, H=2, T=150, d=96, dk=32, dv=48, seed=0):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    return {"x": r(B, T, d), "res": r(B, T, d), "gamma": 1 + 0.1 * r(d), "Wq": r(d, H * dk) / d ** 0.5,
            "Wk": r(d, H * dk) / d, "Wv": r(d, H * dv) / d ** 0.5, "Wa": r(H, d) / d ** 0.5, "Wb": r(H, d) / d ** 0.5,
            "bdt": -2 + 0.1 * r(H), "A": torch.exp(0.1 * r(H)), "Wo": r(H * dv, d) / (H * dv) ** 0.5,
            "gamma2": 1 + 0.1 * r(d), "S0": r(B, H, dk, dv), "c": r(B, T, d)}


def heads(z, H):
    B, T, _ = z.shape
    return z.view(B, T, H, -1).transpose(1, 2).contiguous()


def merge(z):
    B, H, T, n = z.shape
    return z.transpose(1, 2).reshape(B, T, H * n)


def reference(p):
    """The dense layer and the next norm in 64 bits by torch's own derivatives; loss <c, y2>."""
    p = {k: v.double().requires_grad_() for k, v in p.items()}
    norm = lambda h, ga: h / (h.square().mean(-1, keepdim=True) + EPS).sqrt() * ga  # noqa: E731
    H, (B, T, _) = p["A"].shape[0], p["x"].shape
    h = p["x"] + p["res"]
    n = norm(h, p["gamma"])
    q, k, v = (heads(n @ p[w], H) for w in ("Wq", "Wk", "Wv"))
    za = (n @ p["Wa"].t()).transpose(1, 2) + p["bdt"][None, :, None]
    al = torch.exp(-p["A"][None, :, None] * torch.nn.functional.softplus(za))
    be = torch.sigmoid((n @ p["Wb"].t()).transpose(1, 2))
    S, y = p["S0"], []
    for t in range(T):
        S = al[:, :, t, None, None] * S + be[:, :, t, None, None] * k[:, :, t, :, None] * v[:, :, t, None, :]
        y.append((q[:, :, t, :, None] * S).sum(-2))
    o = merge(torch.stack(y, 2)) @ p["Wo"]
    y2 = norm(o + h, p["gamma2"])
    grads = torch.autograd.grad((y2 * p["c"]).sum(), [p[k] for k in ("x", "gamma", "gamma2", "S0", "Wq", "Wv", "bdt", "A")])
    return y2.detach(), dict(zip(("x", "gamma", "gamma2", "S0", "Wq", "Wv", "bdt", "A"), grads))


def program(p):
    """The same through the library; dense products by torch."""
    H = p["A"].shape[0]
    a = sdm.sdm_residual_norm(p["x"], p["gamma"], p["res"], EPS, "f32")
    n, h = a["y"], a["h"]
    q, k, v = (heads(n @ p[w], H) for w in ("Wq", "Wk", "Wv"))
    al, be = sdm.sdm_gates(n, p["Wa"], p["Wb"], p["bdt"], p["A"])
    y, _ = sdm.sdm_dense_scan_forward(q, k, v, al, be, p["S0"])
    my = merge(y)
    b = sdm.sdm_residual_norm(my @ p["Wo"], p["gamma2"], h, EPS, "f32")
    # backwards
    g2 = sdm.sdm_residual_norm_backward(p["c"], b["h"], p["gamma2"], None, EPS)
    dmy = g2["dx"] @ p["Wo"].t()
    s = sdm.sdm_dense_scan_backward(q, k, v, al, be, heads(dmy, H), p["S0"])
    # the gates' inputs, from the gradient to ln alpha and to beta
    za = (n @ p["Wa"].t()).transpose(1, 2) + p["bdt"][None, :, None]
    dza = -p["A"][None, :, None] * torch.sigmoid(za) * s["dlog_alpha"]
    dzb = s["dbeta"] * be * (1 - be)
    dn = merge(s["dq"]) @ p["Wq"].t() + merge(s["dk"]) @ p["Wk"].t() + merge(s["dv"]) @ p["Wv"].t() \
        + dza.transpose(1, 2) @ p["Wa"] + dzb.transpose(1, 2) @ p["Wb"]
    g1 = sdm.sdm_residual_norm_backward(dn.contiguous(), h, p["gamma"], g2["dx"], EPS)
    flat = lambda z: z.reshape(-1, z.shape[-1])  # noqa: E731
    return b["y"], {"x": g1["dx"], "gamma": g1["dgamma"], "gamma2": g2["dgamma"], "S0": s["dS0"],
                    "Wq": flat(n).t() @ flat(merge(s["dq"])), "Wv": flat(n).t() @ flat(merge(s["dv"])),
                    "bdt": dza.sum((0, 2)), "A": (-torch.nn.functional.softplus(za) * s["dlog_alpha"]).sum((0, 2))}


def test_dense_layer_and_its_gradients():
    p = layer()
    want, grads = reference(p)
    y, got = program({k: v.to(DEV) for k, v in p.items()})
    assert (y.cpu().double() - want).abs().max() <= TOL * want.abs().max()
    for k, w in grads.items():
        assert (got[k].cpu().double() - w).abs().max() <= TOL * w.abs().max(), k


def sparse_step(x, wl):
    """Addressing with its balance loss, the training scan, and the write weights' whole gradient."""
    iw, ww, ir, wr = sdm.sdm_address(x["q_w"], x["q_r"], x["subkeys"], x["subkeys"], wl.W, wl.R)
    bal = sdm.sdm_balance_forward(iw, ww, wl.N, x["mask"])
    M = sdm.sdm_state_init(x["M0"], wl.B)
    y, snap = sdm.sdm_scan_forward_save(iw, ww, ir, wr, x["alpha"], x["beta"], x["v"], M)
    g = sdm.sdm_scan_backward(iw, ww, ir, wr, x["alpha"], x["beta"], x["v"], snap, torch.ones_like(y), M, torch.zeros_like(M))
    dwt = sdm.sdm_balance_backward(iw, bal["counts"], bal["tokens"], x["dloss"], x["mask"])
    n = sdm.sdm_residual_norm(y, x["gamma"], None, EPS, "e4m3")
    return {"y": y, "dwt": g["dwt_w"] + dwt, "loss": bal["loss"], "counts": bal["counts"], "mass": bal["mass"],
            "n": n["y"].view(torch.uint8), "scale": n["scale"]}


def test_sparse_layer_with_its_balance_loss_on_streams():
    wl = inputs.get("small", B=2, H=2, T=300)
    x = {k: v.to(DEV) for k, v in inputs.make_inputs(wl).items()}
    x["mask"] = (torch.arange(300, device=DEV)[None] < torch.tensor([[211], [0]], device=DEV)).to(torch.uint8)
    x["dloss"], x["gamma"] = torch.full((2,), 0.01, device=DEV), torch.ones(wl.d_v, device=DEV)
    want = sparse_step(x, wl)
    assert int(want["counts"].sum()) == 211 * 2 * wl.W
    assert torch.allclose(want["mass"].sum(-1), torch.full((2,), 211.0, device=DEV), rtol=1e-5)  # weights sum to 1 a token
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for s in streams:
        with torch.cuda.stream(s):
            got.append(sparse_step(x, wl))
    torch.cuda.synchronize()
    for r in got:
        for k in want:
            assert torch.equal(r[k], want[k]), k


def test_decoding_continues_a_prompt():
    """A prompt in one call, then single tokens with the state in place, against one call over all tokens."""
    p = {k: v.to(DEV) for k, v in layer(T=90).items()}
    H = 2
    n = sdm.sdm_residual_norm(p["x"], p["gamma"], p["res"], EPS, "f32")["y"]
    q, k, v = (heads(n @ p[w], H) for w in ("Wq", "Wk", "Wv"))
    al, be = sdm.sdm_gates(n, p["Wa"], p["Wb"], p["bdt"], p["A"])
    whole, last = sdm.sdm_dense_scan_forward(q, k, v, al, be)
    cut = lambda z, a, b: z[:, :, a:b].contiguous()  # noqa: E731
    y, S = sdm.sdm_dense_scan_forward(*(cut(z, 0, 80) for z in (q, k, v, al, be)))
    ys = [y]
    for t in range(80, 90):
        y, S = sdm.sdm_dense_scan_forward(*(cut(z, t, t + 1) for z in (q, k, v, al, be)), S, S)
        ys.append(y)
    assert (torch.cat(ys, 2) - whole).abs().max() <= TOL * whole.abs().max()
    assert (S - last).abs().max() <= TOL * last.abs().max()


def test_outputs_of_other_names_are_refused():
    """A preallocated tensor under a name that a call does not know would go unused."""
    x = {k: v.to(DEV) for k, v in layer(T=8).items()}
    q, al = torch.zeros((2, 2, 8, 16), device=DEV), torch.ones((2, 2, 8), device=DEV)
    i, w, t = torch.zeros((2, 2, 8, 4), dtype=torch.int32, device=DEV), torch.ones((2, 2, 8, 4), device=DEV), q.new_empty(1)
    for name, call in (("dS", lambda o: sdm.sdm_dense_scan_backward(q, q, q, al, al, q, out=o)),
                       ("dh", lambda o: sdm.sdm_residual_norm_backward(x["c"], x["x"], x["gamma"], out=o)),
                       ("count", lambda o: sdm.sdm_balance_forward(i, w, 16, out=o)),
                       ("scale", lambda o: sdm.sdm_residual_norm(x["x"], x["gamma"], out=o))):
        with pytest.raises(ValueError):
            call({name: t})
        call({})
