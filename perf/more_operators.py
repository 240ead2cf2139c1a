"""The operators of a selective state-space layer, as cases that can be timed and compared.

Such a layer stands beside the sparse and the dense gated ones in a stack. Three families, each
with its plain form (elementary torch operations in 32 bits) and, with ``own`` true, the calls
a program makes of the package:

- ``conv`` / ``conv_backward``: the short causal convolution over time of every channel, in front of
  the recurrence, y_t = act(bias + sum_j w_j x_{t-K+1+j}), with the last K - 1 inputs as its state; and
  its gradients;
- ``scan`` / ``scan_backward``: the selective state-space scan, for each channel d and state n
      delta_t = softplus(dt_t + dt_bias),   h_t = exp(delta_t A) h_{t-1} + delta_t x_t B_t,
      y_t = (C_t h_t + D x_t) silu(z_t),
  and the gradients of all of its inputs;
- ``layer_norm`` / ``layer_norm_backward``: h = x + res, y = (h - mean) / sqrt(var + eps) gamma + bias,
  and its gradients.

Sequences may be packed (``start`` marks tokens that begin one) or padded (``lengths``).
"""
import math

import torch

own = False

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
EPS = 1e-5


# ---------------------------------------------------------------- cases

def listed():
    return [
        # one token of 256 sequences: serving, the states updated in place
        {"name": "conv step", "op": "conv", "B": 256, "H": 1, "T": 1, "d": 2048, "K": 4, "dtype": "bf16", "seq": "none", "step": True},
        # the training forward of a layer twice as wide as the stream, its input the first half of a projection
        {"name": "conv train", "op": "conv", "B": 4, "H": 1, "T": 8192, "d": 2048, "K": 4, "dtype": "bf16", "seq": "none", "step": False},
        # the training backward at the same sizes
        {"name": "conv backward", "op": "conv_backward", "B": 4, "H": 1, "T": 8192, "d": 2048, "K": 4, "dtype": "bf16", "seq": "none"},
        # the keys of a dense gated layer: heads out of a projection, packed sequences, odd sizes, fp32
        {"name": "conv backward f32 packed", "op": "conv_backward", "B": 3, "H": 5, "T": 1003, "d": 77, "K": 3, "dtype": "f32", "seq": "packed"},
        # one token of 256 sequences: serving, the states updated in place
        {"name": "scan step", "op": "scan", "B": 256, "T": 1, "D": 2048, "G": 1, "N": 16, "dtype": "bf16", "seq": "none", "step": True},
        # a training forward or a batch of prompts
        {"name": "scan train", "op": "scan", "B": 4, "T": 8192, "D": 2048, "G": 1, "N": 16, "dtype": "bf16", "seq": "none", "step": False},
        # few long sequences in fp32, padded to the longest, in groups of channels, sizes that fill no tile
        {"name": "scan f32 long padded", "op": "scan", "B": 2, "T": 40001, "D": 520, "G": 2, "N": 24, "dtype": "f32", "seq": "padded", "step": False},
        # a training backward
        {"name": "scan backward", "op": "scan_backward", "B": 4, "T": 4096, "D": 2048, "G": 1, "N": 16, "dtype": "bf16", "seq": "none"},
        # packed sequences in fp32, sizes that fill no tile
        {"name": "scan backward f32 packed", "op": "scan_backward", "B": 3, "T": 1003, "D": 360, "G": 1, "N": 9, "dtype": "f32", "seq": "packed"},
        # the layer width over all tokens of a training step, with the residual stream
        {"name": "layer norm train", "op": "layer_norm", "rows": 32768, "d": 1024, "dtype": "bf16", "out": "bf16", "res": True},
        # a few odd rows in fp32, no residual: latency
        {"name": "layer norm f32 odd", "op": "layer_norm", "rows": 33, "d": 1919, "dtype": "f32", "out": "f32", "res": False},
        # the training backward of the layer width
        {"name": "layer norm backward", "op": "layer_norm_backward", "rows": 32768, "d": 1024, "dtype": "bf16", "dh": True},
    ]


def _logint(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["conv", "conv_backward", "scan", "scan", "scan_backward", "scan_backward", "layer_norm", "layer_norm_backward"])
    seq = rng.choice(["none", "none", "packed", "padded"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op in ("conv", "conv_backward"):
        H = rng.choice([1, 1, 4, 8])
        d = _logint(rng, 32, 4096) // H + 1
        if rng.random() < 0.6:
            d = (d + 7) // 8 * 8
        B = _logint(rng, 1, 8)
        c = {"op": op, "B": B, "H": H, "T": 1, "d": d, "K": rng.choice([2, 3, 4, 4, 8]), "dtype": dtype, "seq": seq}
        if op == "conv":
            c["step"] = rng.random() < 0.3
            if c["step"]:
                c.update(B=_logint(rng, 1, 256), T=rng.choice([1, 1, 1, 2, 3]), seq="none")
                return c
        c["T"] = _logint(rng, 16, max(16, min(16384, (1 << 25) // (B * H * d))))
        return c
    if op in ("scan", "scan_backward"):
        G = rng.choice([1, 1, 1, 2, 4])
        D = G * (_logint(rng, 32, 4096) // G + 1)
        if rng.random() < 0.6:
            D = (D + 63) // 64 * 64
        N = rng.choice([16, 16, 16, 8, 32, 64, rng.randint(1, 64)])
        B = _logint(rng, 1, 8)
        c = {"op": op, "B": B, "T": 1, "D": D, "G": G, "N": N, "dtype": dtype, "seq": seq}
        if op == "scan":
            c["step"] = rng.random() < 0.25
            if c["step"]:
                c.update(B=_logint(rng, 1, 128), T=rng.choice([1, 1, 1, 2, 3]), seq="none")
                return c
        most = (1 << 28) if op == "scan" else (1 << 27)  # elements of all states
        c["T"] = _logint(rng, 30, max(30, min(32768, most // (B * D * max(N, 16)))))
        return c
    d = 128 * rng.randint(1, 64) if rng.random() < 0.6 else _logint(rng, 64, 12000)
    rows = _logint(rng, 1, max(1, min(65536, (1 << 25) // d)))
    c = {"op": op, "rows": rows, "d": d, "dtype": dtype}
    if op == "layer_norm":
        c["out"] = rng.choice(["bf16", "f32"])
        c["res"] = rng.random() < 0.75
    else:
        c["dh"] = rng.random() < 0.75
    return c


# ---------------------------------------------------------------- inputs

def prepare(case, seed):
    dev = "cuda" if torch.cuda.is_available() else "cpu"
    g = torch.Generator(device=dev)
    g.manual_seed(seed)

    def randn(*shape):
        return torch.randn(shape, generator=g, device=dev)

    def rand(*shape):
        return torch.rand(shape, generator=g, device=dev)

    op = case["op"]
    s = {"op": op}
    if op in ("layer_norm", "layer_norm_backward"):
        rows, d, dt = case["rows"], case["d"], DT[case["dtype"]]
        s["gamma"] = 1.0 + 0.1 * randn(d)
        if op == "layer_norm":
            s["bias"] = 0.1 * randn(d)
            s["x"] = (randn(rows, d) * (0.5 + randn(rows, 1).abs()) + randn(rows, 1)).to(dt)
            s["res"] = randn(rows, d).to(dt) if case["res"] else None
            s["out"] = case["out"]
        else:
            s["h"] = (randn(rows, d) * (0.5 + randn(rows, 1).abs()) + randn(rows, 1)).to(dt)
            s["dy"] = randn(rows, d).to(dt)
            s["dh"] = randn(rows, d).to(dt) if case["dh"] else None
        return s
    B, T, dt = case["B"], case["T"], DT[case["dtype"]]
    s["start"] = s["lengths"] = None
    if case["seq"] == "packed":  # sequences of some 200 tokens on end
        s["start"] = (rand(B, T) < 0.005).to(torch.uint8)
    elif case["seq"] == "padded":  # every length from none to all
        s["lengths"] = (rand(B) * (T + 1)).to(torch.int32).clamp_(max=T)
        s["lengths"][-1] = T
    if op in ("conv", "conv_backward"):
        H, d, K = case["H"], case["d"], case["K"]
        if H == 1:  # one half of a projection that gives the gate too
            s["x"] = randn(B, T, 2 * d).to(dt)[..., :d]
            lead = (B,)
        else:  # heads of a projection
            s["x"] = randn(B, T, H * d).to(dt).view(B, T, H, d).transpose(1, 2)
            lead = (B, H)
        s["w"] = randn(*lead[1:], d, K) * K ** -0.5
        s["bias"] = 0.1 * randn(*lead[1:], d)
        s["S0"] = randn(*lead, K - 1, d).to(dt)
        if op == "conv":
            s["step"] = case["step"]
        else:
            s["dy"] = randn(*lead, T, d).to(dt)
            s["dS"] = randn(*lead, K - 1, d).to(dt)
        return s
    D, G, N = case["D"], case["G"], case["N"]
    x = randn(B, T, D)
    s["x"] = (x * torch.sigmoid(x)).to(dt)  # behind the convolution's SiLU
    s["z"] = randn(B, T, 2 * D).to(dt)[..., D:]  # the projection's other half
    low = randn(B, T, 32 + 2 * G * N).to(dt)  # one projection gives the steps' low rank, B and C
    s["B"] = low[..., 32:32 + G * N].view(B, T, G, N)
    s["C"] = low[..., 32 + G * N:].view(B, T, G, N)
    s["dt"] = (0.5 * randn(B, T, D)).to(dt)
    step = torch.exp(rand(D) * math.log(100.0) + math.log(0.001))  # time steps from 0.001 to 0.1
    s["dt_bias"] = step + torch.log(-torch.expm1(-step))
    s["A"] = -torch.arange(1, N + 1, device=dev) * torch.exp(0.1 * randn(D, N))
    s["D"] = 1.0 + 0.1 * randn(D)
    s["S0"] = 0.3 * randn(B, D, N)
    if op == "scan":
        s["step"] = case["step"]
    else:
        s["dy"] = randn(B, T, D).to(dt)
        s["dS"] = 0.1 * randn(B, D, N)
    return s


# ---------------------------------------------------------------- plain forms

def _silu(x):
    return x / (1.0 + torch.exp(-x))


def _on(s, B, T, dev):
    """[B, T]: the tokens that are there."""
    if s["lengths"] is None:
        return torch.ones((B, T), dtype=torch.bool, device=dev)
    return torch.arange(T, device=dev)[None] < s["lengths"][:, None]


def _conv_plain(s, x, w, bias, S0):
    """y and the state behind the last token, of x [B, H, T, d] in 32 bits."""
    B, H, T, d = x.shape
    K = w.shape[-1]
    rows = torch.cat([S0, x], 2)  # rows[t + K - 1] is token t
    run = torch.zeros((B, T + K - 1), dtype=torch.int32, device=x.device)  # sequences begun so far
    if s["start"] is not None:
        run[:, K - 1:] = (s["start"] != 0).to(torch.int32).cumsum(1)
    z = bias[:, None] + torch.zeros_like(x)
    for j in range(K):
        same = (run[:, j:j + T] == run[:, K - 1:])[:, None, :, None]
        z = z + w[:, None, :, j] * torch.where(same, rows[:, :, j:j + T], 0.0)
    on = _on(s, B, T, x.device)[:, None, :, None]
    y = torch.where(on, _silu(z), 0.0)
    n = s["lengths"].long() if s["lengths"] is not None else torch.full((B,), T, device=x.device)
    at = n[:, None] + torch.arange(K - 1, device=x.device)[None]  # rows of the last K - 1 tokens
    same = run.gather(1, at) == run.gather(1, n[:, None] + K - 2)
    S = rows.gather(2, at[:, None, :, None].expand(B, H, K - 1, d)) * same[:, None, :, None]
    return y, S


def _conv_4d(s, *names):
    """The named tensors with their heads (one where there are none)."""
    three = s["x"].dim() == 3
    return [s[n].unsqueeze(0 if n in ("w", "bias") else 1) if three else s[n] for n in names]


def _scan_plain(s, x, dt, A, Bm, Cm, D, z, dt_bias, S0):
    """y and the last state: nc pieces of C tokens side by side, one token of each at a time, then the
    pieces' starting states carried through them."""
    B, T, Dd = x.shape
    G, N = Bm.shape[2:]
    v = dt + dt_bias
    delta = torch.clamp(v, min=0) + torch.log1p(torch.exp(-v.abs()))
    on = _on(s, B, T, x.device)[..., None]
    delta = torch.where(on, delta, 0.0)
    u = delta * x
    C = max(1, math.isqrt(T - 1) + 1)
    nc = (T + C - 1) // C
    pad = nc * C - T

    def cut(t):
        return torch.nn.functional.pad(t.reshape(B, T, -1), (0, 0, 0, pad)).view(B, nc, C, -1)

    dl, ul, bl, cl = cut(delta), cut(u), cut(Bm), cut(Cm)
    go = None if s["start"] is None else 1.0 - cut((s["start"] != 0)[..., None] & on)[..., None].float()

    def decay(i):
        a = torch.exp(dl[:, :, i, :, None] * A)
        return a if go is None else a * go[:, :, i]

    def spread(t, i):  # [B, nc, D, N]
        return t[:, :, i].view(B, nc, G, 1, N).expand(B, nc, G, Dd // G, N).reshape(B, nc, Dd, N)

    h = torch.zeros((B, nc, Dd, N), device=x.device) if nc > 1 else S0[:, None]
    p, ys = torch.ones_like(h), []
    for i in range(C):
        a = decay(i)
        h = a * h + ul[:, :, i, :, None] * spread(bl, i)
        ys.append((h * spread(cl, i)).sum(-1))
        if nc > 1:
            p = p * a
    S = h[:, 0]
    if nc > 1:
        starts = [S0]
        for c in range(nc):
            starts.append(p[:, c] * starts[-1] + h[:, c])
        S, q = starts[-1], torch.stack(starts[:-1], 1)
        for i in range(C):
            q = decay(i) * q
            ys[i] = ys[i] + (q * spread(cl, i)).sum(-1)
    y = torch.stack(ys, 2).view(B, nc * C, Dd)[:, :T]
    return torch.where(on, (y + D * x) * _silu(z), 0.0), S


def _layer_norm_plain(s):
    x = s["x"].float()
    h = x if s["res"] is None else x + s["res"].float()
    c = h - h.mean(-1, keepdim=True)
    y = c * torch.rsqrt(c.square().mean(-1, keepdim=True) + EPS) * s["gamma"] + s["bias"]
    got = {} if s["res"] is None else {"h": h.to(s["res"].dtype)}
    got["y"] = y.to(DT[s["out"]])
    return got


def _layer_norm_backward_plain(s):
    h, dy = s["h"].float(), s["dy"].float()
    c = h - h.mean(-1, keepdim=True)
    r = torch.rsqrt(c.square().mean(-1, keepdim=True) + EPS)
    n, gd = c * r, dy * s["gamma"]
    dx = r * (gd - gd.mean(-1, keepdim=True) - n * (gd * n).mean(-1, keepdim=True))
    if s["dh"] is not None:
        dx = dx + s["dh"].float()
    return {"dx": dx.to(s["h"].dtype), "dgamma": (dy * n).double().sum(0).float(), "dbias": dy.double().sum(0).float()}


# ---------------------------------------------------------------- one pass

SCAN_IN = ("x", "dt", "A", "B", "C", "D", "z", "dt_bias", "S0")


def run(s):
    op = s["op"]
    if own:
        import sparse_memory_linear_amd as sdm
        if op == "conv":
            S = s["S0"] if s["step"] else None  # serving: the states are updated in place
            y, S = sdm.sdm_causal_conv_forward(s["x"], s["w"], s["bias"], "silu", s["S0"], S, start=s["start"], lengths=s["lengths"])
            return {"y": y, "S": S}
        if op == "conv_backward":
            return sdm.sdm_causal_conv_backward(s["dy"], s["x"], s["w"], s["bias"], "silu", s["S0"], s["dS"], start=s["start"], lengths=s["lengths"])
        if op == "scan":
            S = s["S0"] if s["step"] else None
            y, S = sdm.sdm_selective_scan_forward(s["x"], s["dt"], s["A"], s["B"], s["C"], s["D"], s["z"], s["dt_bias"], True,
                                                  s["S0"], S, start=s["start"], lengths=s["lengths"])
            return {"y": y, "S": S}
        if op == "scan_backward":
            return sdm.sdm_selective_scan_backward(s["dy"], s["x"], s["dt"], s["A"], s["B"], s["C"], s["D"], s["z"], s["dt_bias"], True,
                                                   s["S0"], s["dS"], start=s["start"], lengths=s["lengths"])
        if op == "layer_norm":
            return sdm.sdm_residual_layer_norm(s["x"], s["gamma"], s["bias"], s["res"], EPS, s["out"])
        return sdm.sdm_residual_layer_norm_backward(s["dy"], s["h"], s["gamma"], s["dh"], EPS)
    if op == "layer_norm":
        return _layer_norm_plain(s)
    if op == "layer_norm_backward":
        return _layer_norm_backward_plain(s)
    dt = s["x"].dtype
    if op == "conv":
        y, S = _conv_plain(s, *(t.float() for t in _conv_4d(s, "x", "w", "bias", "S0")))
        y, S = y.to(dt).view(s["x"].shape), S.to(dt).view(s["S0"].shape)
        return {"y": y, "S": s["S0"].copy_(S) if s["step"] else S}
    if op == "conv_backward":
        ins = [t.float().detach().requires_grad_() for t in _conv_4d(s, "x", "w", "bias", "S0")]
        y, S = _conv_plain(s, *ins)
        dx, dw, db, dS0 = torch.autograd.grad([y, S], ins, [t.float() for t in _conv_4d(s, "dy", "dS")])
        return {"dx": dx.to(dt).view(s["x"].shape), "dw": dw.view(s["w"].shape), "dbias": db.view(s["bias"].shape),
                "dS0": dS0.to(dt).view(s["S0"].shape)}
    ins = [s[n].float() for n in SCAN_IN]
    if op == "scan":
        y, S = _scan_plain(s, *ins)
        return {"y": y.to(dt), "S": s["S0"].copy_(S) if s["step"] else S}
    ins = [t.detach().requires_grad_() for t in ins]
    y, S = _scan_plain(s, *ins)
    got = torch.autograd.grad([y, S], ins, [s["dy"].float(), s["dS"]])
    return {"d" + n: t.to(dt) if n in ("x", "dt", "z") else t for n, t in zip(SCAN_IN, got)}


def work(case):
    op = case["op"]
    e = 2 if case["dtype"] == "bf16" else 4
    if op in ("conv", "conv_backward"):
        n, K = case["B"] * case["H"] * case["T"] * case["d"], case["K"]
        st = case["B"] * case["H"] * case["d"] * (K - 1) * e
        w = case["H"] * case["d"] * (K + 1) * 4
        if op == "conv":  # x and the state in, y and the state out
            return {"bytes": 2 * n * e + 2 * st + w, "flops": n * (2 * K + 4)}
        # x, dy and the two states in, dx and the state's gradient out
        return {"bytes": 3 * n * e + 3 * st + 2 * w, "flops": n * (6 * K + 10)}
    if op in ("scan", "scan_backward"):
        tok, N = case["B"] * case["T"], case["N"]
        n, st = tok * case["D"], case["B"] * case["D"] * N * 4
        bc = tok * 2 * case["G"] * N
        par = case["D"] * (N + 2) * 4
        if op == "scan":  # x, dt, z, B, C and the state in, y and the state out
            return {"bytes": 4 * n * e + bc * e + 2 * st + par, "flops": n * (7 * N + 10)}
        # also dy and the last state's gradient in; all gradients out; the state is formed again
        return {"bytes": 7 * n * e + bc * (e + 4) + 3 * st + 2 * par, "flops": n * (21 * N + 30)}
    r, d = case["rows"], case["d"]
    if op == "layer_norm":
        return {"bytes": r * d * (e * (3 if case["res"] else 1) + (2 if case["out"] == "bf16" else 4)) + 8 * d, "flops": 8 * r * d}
    return {"bytes": r * d * e * (4 if case["dh"] else 3) + 12 * d, "flops": 13 * r * d}


# ---------------------------------------------------------------- 64 bits, by the definitions

def _exact_conv(s, backward):
    f64 = torch.float64
    x, w, bias, S0 = (t.to(f64) for t in _conv_4d(s, "x", "w", "bias", "S0"))
    B, H, T, d = x.shape
    K = w.shape[-1]
    rows = torch.cat([S0, x], 2)
    if backward:
        dy, dS = (t.to(f64) for t in _conv_4d(s, "dy", "dS"))
        drows, dw, db = torch.zeros_like(rows), torch.zeros_like(w), torch.zeros_like(bias)
    y, S = torch.zeros_like(x), torch.zeros_like(S0)
    for b in range(B):
        n = int(s["lengths"][b]) if s["lengths"] is not None else T
        begins = [0] if s["start"] is None else [0] + [t for t in s["start"][b].nonzero().flatten().tolist() if t < n]
        fresh = s["start"] is not None and T > 0 and n > 0 and bool(s["start"][b, 0])
        for k, t0 in enumerate(begins):
            t1 = begins[k + 1] if k + 1 < len(begins) else n
            if t1 <= t0 and not (k + 1 == len(begins)):
                continue
            # the rows in front of the sequence: the state's in the first one, else zeros
            head = S0[b] if k == 0 and not (fresh and len(begins) == 1) else torch.zeros_like(S0[b])
            ext = torch.cat([head, x[b, :, t0:t1]], 1)
            m = t1 - t0
            win = ext.unfold(1, K, 1)[:, :m] if m else None  # [H, m, d, K]
            if m:
                zz = (win * w[:, None]).sum(-1) + bias[:, None]
                y[b, :, t0:t1] = zz / (1 + (-zz).exp())
            if k + 1 == len(begins):
                S[b] = ext[:, m:m + K - 1]
            if backward:
                dext = torch.zeros_like(ext)
                if m:
                    sg = 1 / (1 + (-zz).exp())
                    dz = dy[b, :, t0:t1] * sg * (1 + zz * (1 - sg))
                    for j in range(K):
                        dext[:, j:j + m] += dz * w[:, None, :, j]
                    dw += (win * dz[..., None]).sum(1)
                    db += dz.sum(1)
                if k + 1 == len(begins):
                    dext[:, m:m + K - 1] += dS[b]
                drows[b, :, K - 1 + t0:K - 1 + t1] += dext[:, K - 1:]
                if k == 0 and not (fresh and len(begins) == 1):
                    drows[b, :, :K - 1] += dext[:, :K - 1]
    if backward:
        return {"dx": drows[:, :, K - 1:].reshape(s["x"].shape), "dw": dw.view(s["w"].shape), "dbias": db.view(s["bias"].shape),
                "dS0": drows[:, :, :K - 1].reshape(s["S0"].shape)}
    return {"y": y.view(s["x"].shape), "S": S.view(s["S0"].shape)}


def _exact_scan(s, backward):
    """Token by token, forwards and, with the states kept, backwards."""
    f64 = torch.float64
    x, dt, A, Bm, Cm, D, z, dt_bias, h = (s[n].to(f64) for n in SCAN_IN)
    B, T, Dd = x.shape
    G, N = Bm.shape[2:]
    v = dt + dt_bias
    delta = torch.where(v > 0, v, 0.0) + (1 + (-v.abs()).exp()).log()
    keep = _on(s, B, T, x.device).to(f64)
    delta = delta * keep[..., None]
    go = torch.ones_like(keep) if s["start"] is None else (s["start"] == 0).to(f64)
    if s["lengths"] is not None:
        go = torch.where(keep > 0, go, 1.0)
    grp = lambda m, t: m[:, t].repeat_interleave(Dd // G, 1)  # noqa: E731  [B, D, N]
    y = torch.zeros_like(x)
    hs = torch.zeros((T + 1, B, Dd, N), dtype=f64, device=x.device) if backward else None
    if backward:
        hs[0] = h
    for t in range(T):
        a = (delta[:, t, :, None] * A).exp() * go[:, t, None, None]
        h = a * h + (delta[:, t] * x[:, t])[..., None] * grp(Bm, t)
        y[:, t] = (h * grp(Cm, t)).sum(-1)
        if backward:
            hs[t + 1] = h
    sg = 1 / (1 + (-z).exp())
    if not backward:
        return {"y": (y + D * x) * z * sg * keep[..., None], "S": h}
    gy = s["dy"].to(f64) * keep[..., None]
    got = {"dz": gy * (y + D * x) * sg * (1 + z * (1 - sg))}
    gy = gy * z * sg
    dx, dde, dA = D * gy, torch.zeros_like(x), torch.zeros_like(A)
    dB, dC = torch.zeros_like(Bm), torch.zeros_like(Cm)
    q = s["dS"].to(f64)
    for t in reversed(range(T)):
        q = q + gy[:, t, :, None] * grp(Cm, t)
        dC[:, t] = (gy[:, t, :, None] * hs[t + 1]).view(B, G, Dd // G, N).sum(2)
        a = (delta[:, t, :, None] * A).exp() * go[:, t, None, None]
        w = q * a * hs[t]
        qb = (q * grp(Bm, t)).sum(-1)
        dde[:, t] = (w * A).sum(-1) + x[:, t] * qb
        dA += (w * delta[:, t, :, None]).sum(0)
        dx[:, t] += delta[:, t] * qb
        dB[:, t] = (q * (delta[:, t] * x[:, t])[..., None]).view(B, G, Dd // G, N).sum(2)
        q = a * q
    ddt = dde * keep[..., None] / (1 + (-v).exp())
    kb = keep[..., None, None]
    got.update(dx=dx, ddt=ddt, dA=dA, dB=dB * kb, dC=dC * kb, dD=(gy * x).sum((0, 1)), ddt_bias=ddt.sum((0, 1)), dS0=q)
    return {"d" + n: got["d" + n] for n in SCAN_IN}


def exact(case, seed):
    s, f64 = prepare(case, seed), torch.float64
    op = case["op"]
    if op in ("conv", "conv_backward"):
        return _exact_conv(s, op == "conv_backward")
    if op in ("scan", "scan_backward"):
        return _exact_scan(s, op == "scan_backward")
    d, ga = case["d"], s["gamma"].to(f64)
    if op == "layer_norm":
        h = s["x"].to(f64) + (s["res"].to(f64) if s["res"] is not None else 0.0)
        m = h.sum(1, keepdim=True) / d
        y = (h - m) / ((h - m).pow(2).sum(1, keepdim=True) / d + EPS).sqrt() * ga + s["bias"].to(f64)
        return {"h": h, "y": y} if s["res"] is not None else {"y": y}
    h, dy = s["h"].to(f64), s["dy"].to(f64)
    m = h.sum(1, keepdim=True) / d
    r = ((h - m).pow(2).sum(1, keepdim=True) / d + EPS).rsqrt()
    n, gd = (h - m) * r, dy * ga
    dx = r * (gd - gd.sum(1, keepdim=True) / d - n * (gd * n).sum(1, keepdim=True) / d)
    if s["dh"] is not None:
        dx = dx + s["dh"].to(f64)
    return {"dx": dx, "dgamma": (dy * n).sum(0), "dbias": dy.sum(0)}
