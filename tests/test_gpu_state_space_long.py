"""The state-space layer's operators where many sequences make tiles and segments long, against 64 bits.

With few sequences a convolution works by tiles of 8 tokens and a scan by segments of 16; with many by up to 32 (backwards
1024) and by hundreds, as in training, in loops that short ones never turn twice. The workspaces' sizes say how long they are.
The same for types that differ between a layer norm's tensors.

Tolerances count roundings of half a step (2^-24 in fp32, 2^-8 for outputs in bf16), as in the tests of the single operators,
with the chains at hand: a convolution's weights' gradient adds a tile's tokens (n additions are n half steps of the
magnitudes at most); a scan's path passes through the decays of one sequence, 4 roundings each, its sum of steps and its
sums for dA, dD and dt_bias are chains of one segment, and 64 for its ends.
"""
import pytest
import torch

import sparse_memory_linear_amd as sdm
import test_gpu_causal_conv as conv_small
import test_gpu_layer_norm as norm_small
import test_gpu_selective_scan as scan_small

DEV = torch.device("cuda:0")
BF, F32 = torch.bfloat16, torch.float32
HALF = {BF: 2.0 ** -8, F32: 2.0 ** -24}
U = 2.0 ** -24


def sequences(B, T, seed, rate):
    """Begins at some `rate` of the tokens and lengths: whole, none, one and any."""
    g = torch.Generator().manual_seed(seed)
    start = (torch.rand((B, T), generator=g) < rate).to(torch.uint8)
    start[0], start[1, 0], start[2, -1] = 0, 1, 1
    lengths = (torch.rand(B, generator=g) * (T + 1)).to(torch.int32)
    lengths[:6] = torch.tensor([T, T, T, 0, 1, T - 1], dtype=torch.int32)
    return start, lengths


def spoil(p, lengths, names, tokens):
    """NaN behind every sequence's last token."""
    n = lengths.to(next(iter(p.values())).device)
    for k in names:
        t = p[k]
        T = t.shape[tokens]
        shape = [1] * t.dim()
        shape[0], shape[tokens] = t.shape[0], T
        on = (torch.arange(T, device=t.device)[None] < n[:, None]).view(shape)
        p[k] = torch.where(on, t, torch.full((), float("nan"), dtype=t.dtype, device=t.device))


# ---------------------------------------------------------------- convolution

def conv_reference(p, start, lengths, tile):
    """Results and tolerances by shifts of whole tensors, with silu."""
    f = lambda t: t.double()  # noqa: E731
    x, w, bias, dy, S0, dS = (f(p[k]) for k in ("x", "w", "bias", "dy", "S0", "dS"))
    B, H, T, d = x.shape
    K = w.shape[-1]
    dev, half = x.device, HALF[p["x"].dtype]
    n = torch.full((B,), T, device=dev) if lengths is None else lengths.to(dev).long()
    on = torch.arange(T, device=dev)[None] < n[:, None]
    x, dy = (torch.where(on[:, None, :, None], t, 0.0) for t in (x, dy))
    run = torch.zeros((B, T + K - 1), dtype=torch.long, device=dev)
    if start is not None:
        run[:, K - 1:] = ((start.to(dev) != 0) & on).long().cumsum(1)
    rows = torch.cat([S0, x], 2)
    same = [(run[:, j:j + T] == run[:, K - 1:])[:, None, :, None].double() for j in range(K)]
    term = [w[:, None, :, j] * rows[:, :, j:j + T] * same[j] for j in range(K)]
    z, mag = bias[:, None] + sum(term), bias.abs()[:, None] + sum(t.abs() for t in term)
    ez, sg, on4 = (K + 1) * U * mag, torch.sigmoid(z), on[:, None, :, None].double()
    y, dv = z * sg, sg * (1 + z * (1 - sg))
    ey = 1.1 * ez + (3 * z.abs() + 14) * U * y.abs() + half * y.abs()
    dz = dy * dv * on4
    edz = dy.abs() * (0.6 * ez + (3 * z.abs() + 14) * U * sg * (1 + z.abs()) + 2 * U * dv.abs())
    drows, trows, dw, tw = torch.zeros_like(rows), torch.zeros_like(rows), torch.zeros_like(w), torch.zeros_like(w)
    chain = tile + K
    for j in range(K):
        wj = w[:, None, :, j]
        drows[:, :, j:j + T] += wj * dz * same[j]
        trows[:, :, j:j + T] += wj.abs() * (edz + (K + 2) * U * dz.abs()) * same[j]
        seen = rows[:, :, j:j + T] * same[j]
        dw[..., j] = (dz * seen).sum((0, 2))
        tw[..., j] = ((edz + chain * U * dz.abs()) * seen.abs()).sum((0, 2))
    at = n[:, None] + torch.arange(K - 1, device=dev)[None]
    kept = (run.gather(1, at) == run.gather(1, n[:, None] + K - 2))[:, None, :, None].double()
    at = at[:, None, :, None].expand(B, H, K - 1, d)
    S = rows.gather(2, at) * kept
    drows.scatter_add_(2, at, dS * kept)
    trows.scatter_add_(2, at, (K + 2) * U * dS.abs() * kept)
    trows += half * (drows.abs() + trows)
    got = {"y": y * on4, "S": S, "dx": drows[:, :, K - 1:], "dS0": drows[:, :, :K - 1], "dw": dw, "dbias": dz.sum((0, 2))}
    tol = {"y": ey, "S": torch.zeros_like(S), "dx": trows[:, :, K - 1:], "dS0": trows[:, :, :K - 1], "dw": tw + U * dw.abs(),
           "dbias": (edz + chain * U * dz.abs()).sum((0, 2)) + U * got["dbias"].abs()}
    return got, tol


@pytest.mark.parametrize("B,H,T,d,K", [(7, 2, 40, 5, 4), (6, 1, 9, 8, 8), (7, 3, 1, 2, 2)])
def test_the_shifted_reference_is_the_looped_one(B, H, T, d, K):
    p = conv_small.make(B, H, T, d, K, F32, T + K)
    start, lengths = sequences(B, T, K, 0.1)
    for st, ln in ((None, None), (start, None), (None, lengths), (start, lengths)):
        want, _ = conv_small.reference(p, "silu", st, ln)
        got, _ = conv_reference(p, st, ln, 8)
        for k in want:
            assert (got[k] - want[k]).abs().max() <= 1e-12 * (1 + want[k].abs().max()), k


def check(got, want, tol):
    for k, w in want.items():
        if k not in got:
            assert k == "dz"
            continue
        bad = ~((got[k].double().reshape(w.shape) - w).abs() <= tol[k] + 1e-37)
        assert not bad.any(), (k, int(bad.sum()), float((got[k].double().reshape(w.shape) - w).abs().max()))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("B,H,T,d,K,tile", [(128, 2, 1100, 13, 4, 72), (128, 1, 1100, 16, 3, 72), (96, 2, 900, 12, 8, 44),
                                            (256, 1, 1030, 24, 4, 132), (2048, 1, 1100, 4, 4, 1024)])
def test_convolution_by_long_tiles(B, H, T, d, K, tile, dtype):
    """Forwards by tiles of 32 (24 in the third case) tokens, backwards by `tile`."""
    need = sdm.sdm_causal_conv_backward_workspace_bytes(B, H, T, d, K)
    assert need == B * -(-T // tile) * (K + 1) * H * d * 4
    p = {k: v.to(DEV) for k, v in conv_small.make(B, H, T, d, K, dtype, T + d).items()}
    start, lengths = sequences(B, T, d, 0.02)
    args = (p["x"], p["w"], p["bias"], "silu", p["S0"])
    for st, ln in ((None, None), (start, None), (start, lengths)):
        want, tol = conv_reference(p, st, ln, tile)
        if ln is not None:
            p = dict(p)
            spoil(p, ln, ("x", "dy"), 2)
            args = (p["x"], *args[1:])
        kw = {"start": None if st is None else st.to(DEV), "lengths": None if ln is None else ln.to(DEV)}
        y, S = sdm.sdm_causal_conv_forward(*args, **kw)
        check({"y": y, "S": S, **sdm.sdm_causal_conv_backward(p["dy"], *args, p["dS"], **kw)}, want, tol)


# ---------------------------------------------------------------- selective scan

def segments(B, T, D, G, N):
    """The fewest tokens a segment, forwards and backwards, that give the workspaces their sizes (selective.hip, selective_bwd.hip)."""
    tiles, nt = B * G * -(-(D // G) // 64), -(-N // 16)
    fwd = sdm.sdm_selective_scan_workspace_bytes(B, T, D, G, N) // (tiles * (nt * 4096 + 256))
    words = sdm.sdm_selective_scan_backward_workspace_bytes(B, T, D, G, N) // 4
    tile = tiles * nt * 1024

    def size(L):
        n = -(-T // L)
        return n * (3 * tile + tiles * 64 + nt * tiles * 128) + n * (L // 8) * (tile + tiles * 64) + tiles * T * nt * 32

    return -(-T // max(fwd, 1)), min(L for L in range(16, T + 8, 8) if size(L) == words)


def scan_reference(p, start, lengths, L):
    B, T, _ = p["x"].shape
    with DEV:
        n = torch.full((B,), T) if lengths is None else lengths.to(DEV).clamp(0, T)
        keep = (torch.arange(T)[None] < n[:, None]).double()
        go = torch.ones_like(keep)
        if start is not None:
            go = torch.where((start.to(DEV) != 0) & (keep > 0), 0.0, 1.0).double()
        # the longest sequence
        last = torch.where(go == 0, torch.arange(T)[None], 0).cummax(1).values
        path = int((torch.arange(T)[None] - last).max()) + 1
        want, mag = (scan_small.formulas(p, True, keep, go, m) for m in (False, True))
    half = HALF[p["x"].dtype]
    tol = {k: (4 * path + L + 64) * U * mag[k] * 1.01 + (half if k in ("y", "dx", "ddt", "dz") else U) * 1.01 * want[k].abs() for k in want}
    return want, tol


# whole sequences in one launch forwards (no workspace): 96 x 16 groups. The others are cut, forwards by `fwd` tokens or more.
@pytest.mark.gpu
@pytest.mark.parametrize("B,T,D,G,N,fwd,bwd,dtype", [(64, 2100, 70, 1, 9, 40, 72, F32), (64, 2100, 70, 1, 9, 40, 72, BF),
                                                     (32, 2400, 130, 2, 20, 80, 152, F32), (24, 1100, 16, 16, 40, 138, 280, BF),
                                                     (24, 1100, 16, 16, 40, 138, 280, F32), (96, 300, 16, 16, 5, 300, 104, F32),
                                                     (96, 300, 16, 16, 5, 300, 104, BF)])
def test_scan_by_long_segments(B, T, D, G, N, fwd, bwd, dtype):
    f, b = segments(B, T, D, G, N)
    assert (f, b) == (fwd, bwd)
    p = {k: v.to(DEV) for k, v in scan_small.make(B, T, D, G, N, dtype, T + D).items()}
    start, lengths = sequences(B, T, D, 0.02)
    start[0] = start[3]
    start[0, bwd + 24], start[0, bwd + 71] = 1, 1  # in chunks of a segment behind its second
    for st, ln, less in ((None, None, 6.0), (start, None, 0.0), (start, lengths, 0.0)):
        q = dict(p, dt=p["dt"] - less)  # (small steps where no sequence begins: what the carries bring counts)
        if ln is None:
            want, tol = scan_reference(q, st, ln, max(bwd, fwd))
        else:
            on = (torch.arange(T, device=DEV)[None] < ln.to(DEV)[:, None]).double()
            names = ("x", "dt", "z", "B", "C", "dy")
            zero = {k: torch.where(on.view(B, T, *[1] * (q[k].dim() - 2)) > 0, q[k], torch.zeros_like(q[k])) for k in names}
            want, tol = scan_reference(dict(q, **zero), st, ln, max(bwd, fwd))
            spoil(q, ln, names, 1)
        kw = {"start": None if st is None else st.to(DEV), "lengths": None if ln is None else ln.to(DEV)}
        args = (q["x"], q["dt"], q["A"], q["B"], q["C"], q["D"], q["z"], q["dt_bias"], True, q["S0"])
        y, S = sdm.sdm_selective_scan_forward(*args, **kw)
        check({"y": y, "S": S, **sdm.sdm_selective_scan_backward(q["dy"], *args, q["dS"], **kw)}, want, tol)
        del want, tol


# ---------------------------------------------------------------- layer norm

MIXED = [(1, 1), (33, 1024), (4, 1919), (3, 5120), (2, 8200), (2, 16384), (1300, 96), (70, 260)]


@pytest.mark.gpu
@pytest.mark.parametrize("gt,ht", [(BF, F32), (F32, BF)], ids=["bf16 over f32", "f32 over bf16"])
@pytest.mark.parametrize("rows,d", MIXED)
def test_layer_norm_backward_of_two_types(rows, d, gt, ht):
    h0, _, gamma, _, _, _ = norm_small.make(rows, d, ht, rows + d)
    _, dh, _, _, dy, _ = norm_small.make(rows, d, gt, rows + 2 * d)
    h, c, ec, r, er, _ = norm_small.parts(h0, None)
    DY, GA = dy.double(), gamma.double()
    n, gd = c * r, GA * DY
    en = ec * r + c.abs() * er + U * n.abs()
    mean = lambda t: t.mean(-1, keepdim=True)  # noqa: E731
    want = r * (gd - mean(gd) - n * mean(gd * n))
    inner = gd.abs() + mean(gd.abs()) + n.abs() * mean((gd * n).abs())
    e = er * inner + r * ((d + 8) * U * inner + en * mean((gd * n).abs()) + n.abs() * mean(gd.abs() * en))
    per = -(-rows // 256) + 64
    for t in (None, dh):
        w = want if t is None else want + t.double()
        got = sdm.sdm_residual_layer_norm_backward(dy.to(DEV), h0.to(DEV), gamma.to(DEV), None if t is None else t.to(DEV), 1e-5)
        assert got["dx"].dtype == gt
        mag = w.abs() + (t.double().abs() if t is not None else 0)
        assert ((got["dx"].cpu().double() - w).abs() <= 1.01 * e + 2 * U * mag + HALF[gt] * w.abs() * 1.001 + 1e-37).all()
        dg, db = (DY * n).sum(0), DY.sum(0)
        assert ((got["dgamma"].cpu().double() - dg).abs() <= 1.01 * (DY.abs() * en).sum(0) + (per + 4) * U * (DY * n).abs().sum(0) + 1e-37).all()
        assert ((got["dbias"].cpu().double() - db).abs() <= (per + 4) * U * DY.abs().sum(0) + 1e-37).all()


@pytest.mark.gpu
@pytest.mark.parametrize("out", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("xt,rt", [(BF, F32), (F32, BF)], ids=["bf16 onto f32", "f32 onto bf16"])
@pytest.mark.parametrize("rows,d", MIXED)
def test_layer_norm_of_two_types(rows, d, xt, rt, out):
    x, _, gamma, bias, _, _ = norm_small.make(rows, d, xt, rows + d)
    _, res, _, _, _, _ = norm_small.make(rows, d, rt, rows + 2 * d)
    h, c, ec, r, er, mag = norm_small.parts(x, res)
    n = c * r
    y = n * gamma.double() + bias.double()
    ey = (ec * r + c.abs() * er + U * n.abs()) * gamma.double().abs() + 2 * U * (n.abs() * gamma.double().abs() + bias.double().abs())
    got = sdm.sdm_residual_layer_norm(x.to(DEV), gamma.to(DEV), bias.to(DEV), res.to(DEV), 1e-5, {BF: "bf16", F32: "f32"}[out])
    assert got["h"].dtype == rt and got["y"].dtype == out
    assert ((got["h"].cpu().double() - h).abs() <= HALF[rt] * h.abs() * (1 + 1e-6) + U * mag + 1e-38).all()
    assert ((got["y"].cpu().double() - y).abs() <= HALF[out] * y.abs() + 1.01 * ey + 1e-37).all()
