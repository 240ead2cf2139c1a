"""The operators of a layer stack around the sparse memory, as cases that can be timed and compared.

Three families, each with its plain form (elementary torch operations in 32 bits, in 64 where
32 lose what matters) and, with ``own`` true, the calls a program makes of the package:

- ``scan`` / ``scan_backward``: the dense gated recurrence
      S_t = alpha_t S_{t-1} + beta_t k_t (x) v_t,   y_t = q_t S_t
  over [B, H, T] tokens with the scan's gates, and its gradients (the gates' as d/d ln alpha
  and d/d beta);
- ``norm`` / ``norm_backward``: h = x + res, y = h / sqrt(mean h^2 + eps) * gamma, stored in
  fp32, bf16, or e4m3 with one scale per row or per group of columns; and its gradients;
- ``balance``: per-head slot counts and weight mass of an addressing result, the balance loss
  N sum_i f_i P_i (f_i the share of selections, P_i the mean weight of slot i) over the tokens a
  mask keeps, and its gradient to the weights.
"""
import math

import torch

own = False

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
EPS = 1e-6


# ---------------------------------------------------------------- cases

def listed():
    return [
        # one token for each of 256 sequences: serving, the states updated in place
        {"name": "scan step", "op": "scan", "B": 256, "H": 8, "T": 1, "dk": 128, "dv": 128, "dtype": "bf16", "mu": 2.0, "step": True},
        # the GDN-matched layer: a training forward
        {"name": "scan train", "op": "scan", "B": 4, "H": 8, "T": 8192, "dk": 128, "dv": 128, "dtype": "bf16", "mu": 2.0, "step": False},
        # one long sequence: few streams, many tokens
        {"name": "scan long", "op": "scan", "B": 1, "H": 8, "T": 131072, "dk": 128, "dv": 128, "dtype": "bf16", "mu": 4.0, "step": False},
        # the small fp32 layer with a length that fills no tile
        {"name": "scan f32 ragged", "op": "scan", "B": 4, "H": 4, "T": 4001, "dk": 64, "dv": 64, "dtype": "f32", "mu": 2.0, "step": False},
        # the GDN-matched layer: a training backward
        {"name": "scan backward", "op": "scan_backward", "B": 4, "H": 8, "T": 8192, "dk": 128, "dv": 128, "dtype": "bf16", "mu": 2.0},
        # fp32 training with head sizes and a length that fill no tile
        {"name": "scan backward f32 ragged", "op": "scan_backward", "B": 3, "H": 4, "T": 1003, "dk": 96, "dv": 72, "dtype": "f32", "mu": 2.0},
        # a few rows of the layer width, written in 8 bits for the next projection: latency
        {"name": "norm step e4m3", "op": "norm", "rows": 8, "d": 1024, "dtype": "bf16", "out": "e4m3", "group": 0, "res": True},
        # the layer width over all tokens of the GDN-matched layer, with a scale per 128 columns
        {"name": "norm train e4m3", "op": "norm", "rows": 32768, "d": 1024, "dtype": "bf16", "out": "e4m3", "group": 128, "res": True},
        # a wide fp32 stream, odd sizes, no residual
        {"name": "norm f32 odd", "op": "norm", "rows": 4099, "d": 1919, "dtype": "f32", "out": "f32", "group": 0, "res": False},
        # the training backward at the same rows
        {"name": "norm backward", "op": "norm_backward", "rows": 32768, "d": 1024, "dtype": "bf16", "dh": True},
        # the write slots of the GDN-matched layer, all tokens kept
        {"name": "balance train", "op": "balance", "B": 4, "H": 8, "T": 8192, "K": 64, "N": 65536, "mask": False},
        # a padded batch of one head's large table
        {"name": "balance padded", "op": "balance", "B": 7, "H": 1, "T": 9001, "K": 8, "N": 262144, "mask": True},
    ]


def _logint(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["scan", "scan", "scan_backward", "norm", "norm_backward", "balance"])
    if op in ("scan", "scan_backward"):
        dk = 8 * rng.randint(4, 32) if rng.random() < 0.5 else rng.choice([64, 128, 256])
        dv = 8 * rng.randint(4, 32) if rng.random() < 0.5 else rng.choice([64, 128, 256])
        dtype = rng.choice(["bf16", "bf16", "f32"])
        H = rng.choice([1, 2, 4, 5, 8, 16])
        most = (1 << 17) if op == "scan" else (1 << 15)  # token-heads of the drawn call
        c = {"op": op, "B": 1, "H": H, "T": 1, "dk": dk, "dv": dv, "dtype": dtype, "mu": rng.choice([2.0, 3.0, 4.0])}
        if op == "scan":
            c["step"] = rng.random() < 0.25
            if c["step"]:
                c["B"] = _logint(rng, 1, 128)
                c["T"] = rng.choice([1, 1, 1, 2, 3])
                return c
        c["B"] = _logint(rng, 1, 8)
        c["T"] = _logint(rng, 30, max(30, most // (c["B"] * H)))
        return c
    if op in ("norm", "norm_backward"):
        d = 128 * rng.randint(1, 64) if rng.random() < 0.6 else _logint(rng, 64, 12000)
        rows = _logint(rng, 1, max(1, min(65536, (1 << 27) // d // 4)))
        c = {"op": op, "rows": rows, "d": d, "dtype": rng.choice(["bf16", "bf16", "f32"])}
        if op == "norm":
            c["out"] = rng.choice(["e4m3", "bf16", "f32"])
            c["group"] = rng.choice([0, 128, 64]) if c["out"] == "e4m3" and d % 128 == 0 else 0
            c["res"] = rng.random() < 0.75
        else:
            c["dh"] = rng.random() < 0.75
        return c
    n = 16 * rng.randint(1, 32)
    K = rng.choice([1, 8, 16, 33, 64])
    H = rng.choice([1, 2, 4, 8])
    B = _logint(rng, 1, 8)
    return {"op": op, "B": B, "H": H, "T": _logint(rng, 1, max(1, (1 << 23) // (B * H * K))), "K": min(K, n * n),
            "N": n * n, "mask": rng.random() < 0.5}


# ---------------------------------------------------------------- inputs

def prepare(case, seed):
    dev = "cuda" if torch.cuda.is_available() else "cpu"
    g = torch.Generator(device=dev)
    g.manual_seed(seed)

    def randn(*shape):
        return torch.randn(shape, generator=g, device=dev)

    op = case["op"]
    s = {"op": op}
    if op in ("scan", "scan_backward"):
        B, H, T, dk, dv = (case[n] for n in ("B", "H", "T", "dk", "dv"))
        dt = DT[case["dtype"]]
        # keys of unit length, queries scaled by dk^-1/2: what the projections of such a layer give
        k = randn(B, H, T, dk)
        s["k"] = (k / k.square().sum(-1, keepdim=True).sqrt()).to(dt)
        s["q"] = (randn(B, H, T, dk) * dk ** -0.5).to(dt)
        s["v"] = randn(B, H, T, dv).to(dt)
        s["alpha"] = torch.sigmoid(randn(B, H, T) * 0.5 + case["mu"])
        s["beta"] = torch.sigmoid(randn(B, H, T))
        s["S0"] = randn(B, H, dk, dv)
        if op == "scan":
            s["step"] = case["step"]
        else:
            s["dy"] = randn(B, H, T, dv)
            s["dS"] = randn(B, H, dk, dv) * 0.1
    elif op in ("norm", "norm_backward"):
        rows, d, dt = case["rows"], case["d"], DT[case["dtype"]]
        s["gamma"] = 1.0 + 0.1 * randn(d)
        if op == "norm":
            s["x"] = (randn(rows, d) * (0.5 + randn(rows, 1).abs())).to(dt)
            s["res"] = randn(rows, d).to(dt) if case["res"] else None
            s["out"], s["group"] = case["out"], case["group"]
        else:
            s["h"] = (randn(rows, d) * (0.5 + randn(rows, 1).abs())).to(dt)
            s["dy"] = randn(rows, d).to(dt)
            s["dh"] = randn(rows, d).to(dt) if case["dh"] else None
    else:
        B, H, T, K, N = (case[n] for n in ("B", "H", "T", "K", "N"))
        u = torch.rand((B, H, T, K), generator=g, device=dev)
        s["idx"] = (N * u * u).to(torch.int32).clamp_(0, N - 1)  # some slots are chosen far more often
        s["wt"] = torch.softmax(randn(B, H, T, K), -1)
        s["N"] = N
        if case["mask"]:  # padded: each sequence keeps its first tokens, the first one none
            keep = (torch.rand((B, 1), generator=g, device=dev) * T).long()
            keep[0] = 0 if B > 1 else T
            s["mask"] = (torch.arange(T, device=dev)[None] < keep).to(torch.uint8)
        else:
            s["mask"] = None
        s["dloss"] = 0.01 * (1.0 + torch.rand((H,), generator=g, device=dev))
    return s


# ---------------------------------------------------------------- plain forms

def _carry(U, la):
    """X_c = exp(la_c) X_{c-1} + U_c (X_{-1} = 0) along dim 1, U [n, c, m], la [n, c] in 64 bits:
    groups of 64 by a decay matrix, the groups' ends by the same step."""
    n, c, m = U.shape
    G = 64
    pad = -c % G
    U = torch.nn.functional.pad(U, (0, 0, 0, pad)).view(n, -1, G, m)
    la = torch.nn.functional.pad(la, (0, pad)).view(n, -1, G)
    cs = la.cumsum(-1)
    keep = torch.ones(G, G, dtype=torch.bool, device=U.device).tril()
    D = (cs[..., :, None] - cs[..., None, :]).masked_fill(~keep, -math.inf).exp().float()
    X = D @ U
    if U.shape[1] > 1:
        ends = _carry(X[:, :, -1], cs[..., -1])
        before = torch.nn.functional.pad(ends, (0, 0, 1, 0))[:, :-1]
        X = X + cs.exp().float()[..., None] * before[:, :, None]
    return X.reshape(n, -1, m)[:, :c]


def _scan_plain(q, k, v, la, beta, S0):
    """y and the last state, chunks of up to 64 tokens; la = ln alpha in 64 bits."""
    B, H, T, dk = q.shape
    dv, C, n = v.shape[-1], min(64, T), B * H
    pad = -T % C
    q, k, v = (torch.nn.functional.pad(x.reshape(n, T, -1), (0, 0, 0, pad)).view(n, -1, C, x.shape[-1]) for x in (q, k, v))
    beta = torch.nn.functional.pad(beta.reshape(n, T), (0, pad)).view(n, -1, C)
    cs = torch.nn.functional.pad(la.reshape(n, T), (0, pad)).view(n, -1, C).cumsum(-1)
    keep = torch.ones(C, C, dtype=torch.bool, device=q.device).tril()
    D = (cs[..., :, None] - cs[..., None, :]).masked_fill(~keep, -math.inf).exp().float()
    P = (q @ k.transpose(-1, -2).contiguous()) * D * beta[..., None, :]
    to_end = (cs[..., -1:] - cs).exp().float() * beta
    U = (k * to_end[..., None]).transpose(-1, -2).contiguous() @ v
    S0 = S0.reshape(n, 1, dk * dv)
    chunk = cs[..., -1]
    X = _carry(U.reshape(n, -1, dk * dv), chunk) + chunk.cumsum(-1).exp().float()[..., None] * S0
    start = torch.cat([S0, X[:, :-1]], 1).view(n, -1, dk, dv)
    y = P @ v + cs.exp().float()[..., None] * (q @ start)
    return y.reshape(n, -1, dv)[:, :T].reshape(B, H, T, dv), X[:, -1].reshape(B, H, dk, dv)


def _scan_backward_plain(s):
    q, k, v = (s[n].float().requires_grad_() for n in ("q", "k", "v"))
    la = s["alpha"].double().log().requires_grad_()
    beta, S0 = (s[n].detach().clone().requires_grad_() for n in ("beta", "S0"))
    y, S = _scan_plain(q, k, v, la, beta, S0)
    dq, dk, dv, dla, db, dS0 = torch.autograd.grad([y, S], [q, k, v, la, beta, S0], [s["dy"], s["dS"]])
    return {"dq": dq, "dk": dk, "dv": dv, "dlog_alpha": dla.float(), "dbeta": db, "dS0": dS0}


def _norm_plain(s):
    x = s["x"].float()
    h = x if s["res"] is None else x + s["res"].float()
    y = h * torch.rsqrt(h.square().mean(-1, keepdim=True) + EPS) * s["gamma"]
    got = {} if s["res"] is None else {"h": h.to(s["res"].dtype)}
    if s["out"] == "e4m3":
        yg = y.view(y.shape[0], -1, s["group"] or y.shape[1])
        scale = yg.abs().amax(-1) / 448.0
        got["y"] = (yg / scale[..., None]).to(torch.float8_e4m3fn).view(y.shape)
        got["scale"] = scale
    else:
        got["y"] = y.to(DT[s["out"]])
    return got


def _norm_backward_plain(s):
    h, dy = s["h"].float(), s["dy"].float()
    r = torch.rsqrt(h.square().mean(-1, keepdim=True) + EPS)
    n, gd = h * r, dy * s["gamma"]
    dx = r * (gd - n * (gd * n).mean(-1, keepdim=True))
    if s["dh"] is not None:
        dx = dx + s["dh"].float()
    return {"dx": dx.to(s["h"].dtype), "dgamma": (dy * n).double().sum(0).float()}


def _balance_plain(s):
    idx, wt, N = s["idx"], s["wt"], s["N"]
    B, H, T, K = idx.shape
    at = idx.long() + N * torch.arange(H, device=idx.device)[None, :, None, None]
    keep = torch.ones((B, 1, T, 1), device=idx.device) if s["mask"] is None else s["mask"].view(B, 1, T, 1).float()
    tokens = keep.sum().to(torch.int32)
    counts = torch.zeros(H * N, dtype=torch.int32, device=idx.device)
    counts.index_add_(0, at.flatten(), keep.expand_as(wt).to(torch.int32).flatten())
    mass = torch.zeros(H * N, dtype=torch.float64, device=idx.device)
    mass.index_add_(0, at.flatten(), (wt * keep).double().flatten())
    n = tokens.double().clamp_min(1.0)
    f, P = counts.view(H, N) / (n * K), mass.view(H, N) / n
    loss = N * (f * P).sum(-1)
    dwt = (s["dloss"].double() * (N / n))[None, :, None, None] * f.flatten()[at] * keep
    return {"counts": counts.view(H, N), "mass": mass.view(H, N).float(), "tokens": tokens.view(1), "loss": loss.float(), "dwt": dwt.float()}


# ---------------------------------------------------------------- one pass

def run(s):
    op = s["op"]
    if own:
        import sparse_memory_linear_amd as sdm
        if op == "scan":
            S = s["S0"] if s["step"] else None  # serving: the states are updated in place
            y, S = sdm.sdm_dense_scan_forward(s["q"], s["k"], s["v"], s["alpha"], s["beta"], s["S0"], S)
            return {"y": y, "S": S}
        if op == "scan_backward":
            return sdm.sdm_dense_scan_backward(s["q"], s["k"], s["v"], s["alpha"], s["beta"], s["dy"], s["S0"], s["dS"])
        if op == "norm":
            return sdm.sdm_residual_norm(s["x"], s["gamma"], s["res"], EPS, s["out"], s["group"])
        if op == "norm_backward":
            return sdm.sdm_residual_norm_backward(s["dy"], s["h"], s["gamma"], s["dh"], EPS)
        got = sdm.sdm_balance_forward(s["idx"], s["wt"], s["N"], s["mask"])
        got["dwt"] = sdm.sdm_balance_backward(s["idx"], got["counts"], got["tokens"], s["dloss"], s["mask"])
        return got
    if op == "scan":
        y, S = _scan_plain(s["q"].float(), s["k"].float(), s["v"].float(), s["alpha"].double().log(), s["beta"], s["S0"])
        if s["step"]:
            S = s["S0"].copy_(S)
        return {"y": y, "S": S}
    if op == "scan_backward":
        return _scan_backward_plain(s)
    if op == "norm":
        return _norm_plain(s)
    if op == "norm_backward":
        return _norm_backward_plain(s)
    return _balance_plain(s)


def work(case):
    op = case["op"]
    if op in ("scan", "scan_backward"):
        n, dk, dv = case["B"] * case["H"], case["dk"], case["dv"]
        e = 2 if case["dtype"] == "bf16" else 4
        tok, st = n * case["T"], n * dk * dv * 4
        if op == "scan":  # q, k, v, the two gates and the state in; y and the state out
            return {"bytes": tok * ((2 * dk + dv) * e + 8 + 4 * dv) + 2 * st, "flops": 4 * tok * dk * dv}
        # also dy and the last state's gradient in; all gradients out; the state is formed again
        return {"bytes": tok * ((2 * dk + dv) * e + 8 + 4 * dv + (2 * dk + dv) * 4 + 8) + 3 * st, "flops": 10 * tok * dk * dv}
    if op in ("norm", "norm_backward"):
        r, d = case["rows"], case["d"]
        e = 2 if case["dtype"] == "bf16" else 4
        if op == "norm":
            o = {"f32": 4, "bf16": 2, "e4m3": 1}[case["out"]]
            sc = 4 * r * (d // case["group"] if case["group"] else 1) if case["out"] == "e4m3" else 0
            return {"bytes": r * d * (e * (3 if case["res"] else 1) + o) + 4 * d + sc, "flops": 6 * r * d}
        return {"bytes": r * d * e * (4 if case["dh"] else 3) + 8 * d, "flops": 10 * r * d}
    n = case["B"] * case["H"] * case["T"] * case["K"]
    m = case["B"] * case["T"] if case["mask"] else 0
    return {"bytes": n * 12 + case["H"] * case["N"] * 8 + m, "flops": 4 * n}


# ---------------------------------------------------------------- 64 bits, by the definitions

def _exact_scan(s, backward):
    """The recurrence as sums over pairs of tokens, for one stream and one block of rows at a time:
    y_t = A_t q_t S0 + sum_{s<=t} D_ts beta_s (q_t.k_s) v_s, D_ts = alpha_{s+1} .. alpha_t."""
    B, H, T, dk = s["q"].shape
    dv, n, f64 = s["v"].shape[-1], B * H, torch.float64
    q, k, v = (s[x].reshape(n, T, -1).to(f64) for x in ("q", "k", "v"))
    be, S0 = s["beta"].reshape(n, T).to(f64), s["S0"].reshape(n, dk, dv).to(f64)
    cs = s["alpha"].reshape(n, T).to(f64).log().cumsum(-1)
    if backward:
        dy, dS = s["dy"].reshape(n, T, dv).to(f64), s["dS"].reshape(n, dk, dv).to(f64)
        dq, dk_, dv_ = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
        dS0, X = torch.zeros_like(S0), torch.zeros(n, T, dtype=f64, device=q.device)
        dbe = torch.zeros_like(X)
    else:
        y, S = torch.zeros_like(v), torch.zeros_like(S0)
    R = 2048
    for i in range(n):
        A, E = cs[i].exp(), (cs[i, -1] - cs[i]).exp()  # decay from the start, and to the end
        kb = be[i, :, None] * k[i]
        if not backward:
            S[i] = A[-1] * S0[i] + (kb * E[:, None]).t() @ v[i]
        else:
            row, col = torch.zeros_like(A), torch.zeros_like(A)
            dS0[i] = A[-1] * dS[i] + (q[i] * A[:, None]).t() @ dy[i]
            dkb = E[:, None] * (v[i] @ dS[i].t())       # d/d(beta_s k_s)
            dv_[i] = E[:, None] * (kb @ dS[i])
            into = (kb * dkb).sum(-1)                     # passes from s into the last state
            out = A * (q[i] * (dy[i] @ S0[i].t())).sum(-1)  # passes from the first state to t
        for r in range(0, T, R):
            e = min(T, r + R)
            t = torch.arange(r, e, device=q.device)
            D = cs[i, r:e, None] - cs[i, None, :e]
            D = D.masked_fill_(torch.arange(e, device=q.device)[None] > t[:, None], -math.inf).exp_()
            if not backward:
                y[i, r:e] = A[r:e, None] * (q[i, r:e] @ S0[i]) + ((q[i, r:e] @ kb[:e].t()) * D) @ v[i, :e]
                continue
            P, W = (q[i, r:e] @ kb[:e].t()) * D, (dy[i, r:e] @ v[i, :e].t()) * D
            dq[i, r:e] = A[r:e, None] * (dy[i, r:e] @ S0[i].t()) + W @ kb[:e]
            dkb[:e] += W.t() @ q[i, r:e]
            dv_[i, :e] += P.t() @ dy[i, r:e]
            Z = P * (dy[i, r:e] @ v[i, :e].t())
            Z = Z.masked_fill_(torch.arange(e, device=q.device)[None] == t[:, None], 0.0)
            row[r:e] += Z.sum(1)
            col[:e] += Z.sum(0)
        if backward:
            dk_[i], dbe[i] = be[i, :, None] * dkb, (k[i] * dkb).sum(-1)
            # alpha_t is crossed by pairs s < t <= u, by what comes from the first state to u >= t, by what goes
            # from s < t into the last state, and by the first state's way into the last
            back = lambda z: z.flip(0).cumsum(0).flip(0)  # noqa: E731
            X[i] = back(row) - back(col) + back(out) + (into.cumsum(0) - into) + A[-1] * (dS[i] * S0[i]).sum()
    if backward:
        return {"dq": dq.view_as(s["q"]), "dk": dk_.view_as(s["k"]), "dv": dv_.view_as(s["v"]), "dlog_alpha": X.view(B, H, T),
                "dbeta": dbe.view(B, H, T), "dS0": dS0.view(B, H, dk, dv)}
    return {"y": y.view(B, H, T, dv), "S": S.view(B, H, dk, dv)}


def exact(case, seed):
    s, f64 = prepare(case, seed), torch.float64
    op = case["op"]
    if op in ("scan", "scan_backward"):
        return _exact_scan(s, op == "scan_backward")
    if op == "norm":
        h = s["x"].to(f64) + (s["res"].to(f64) if s["res"] is not None else 0.0)
        y = h / (h.pow(2).sum(1, keepdim=True) / case["d"] + EPS).sqrt() * s["gamma"].to(f64)
        got = {"h": h} if s["res"] is not None else {}
        if case["out"] == "e4m3":
            w = case["group"] or case["d"]
            scale = torch.stack([p.abs().max(1).values for p in y.split(w, 1)], 1) / 448.0
            got["scale"], y = scale, y / scale.repeat_interleave(w, 1)
        got["y"] = y
        return got
    if op == "norm_backward":
        h, dy, ga = s["h"].to(f64), s["dy"].to(f64), s["gamma"].to(f64)
        m = h.pow(2).sum(1, keepdim=True) / case["d"] + EPS
        dx = dy * ga / m.sqrt() - h * (dy * ga * h).sum(1, keepdim=True) / (case["d"] * m.pow(1.5))
        if s["dh"] is not None:
            dx = dx + s["dh"].to(f64)
        return {"dx": dx, "dgamma": (dy * h / m.sqrt()).sum(0)}
    B, H, T, K, N = (case[n] for n in ("B", "H", "T", "K", "N"))
    idx, wt = s["idx"].long(), s["wt"].to(f64)
    on = torch.ones(B, T, dtype=torch.bool, device=wt.device) if s["mask"] is None else s["mask"].bool()
    n = int(on.sum())
    counts, mass = [], []
    dwt = torch.zeros_like(wt)
    for h in range(H):
        i, w = idx[:, h][on].flatten(), wt[:, h][on].flatten()
        counts.append(torch.bincount(i, minlength=N))
        mass.append(torch.bincount(i, weights=w, minlength=N))
        dwt[:, h][on] = s["dloss"][h].to(f64) * N * counts[-1][i].to(f64).view(-1, K) / (n * K) / max(n, 1) if n else 0.0
    counts, mass = torch.stack(counts), torch.stack(mass)
    loss = N * (counts.to(f64) * mass).sum(1) / max(n * K, 1) / max(n, 1)
    return {"counts": counts.to(torch.int32), "mass": mass, "tokens": torch.tensor([n], dtype=torch.int32, device=wt.device), "loss": loss, "dwt": dwt}
