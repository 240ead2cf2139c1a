"""Layer norm with the residual's addition and its gradients against 64 bits.

Tolerances count roundings of half a step: sums over d in some tree or chain, at most n = d additions (2^-24
each, of the terms' magnitudes). The mean is off by (d + 2) half steps of mean |h|, which is also what that puts on every
h - m; outputs in bf16 add 2^-8 relative, e4m3 half a step of 2^-4 relative.
"""
import pytest
import torch

import sparse_memory_linear_amd as sdm

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
BF, F32, F8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
HALF = {BF: 2.0 ** -8, F32: 2.0 ** -24, F8: 2.0 ** -4}
U = 2.0 ** -24
EPS = 1e-5
SIZES = [(1, 1), (2, 7), (5, 64), (3, 100), (8, 512), (33, 1024), (4, 1919), (3, 2048), (5, 2052), (2, 4097),
         (3, 5120), (2, 8200), (2, 8192), (1, 12001), (2, 16384), (1, 16383), (1300, 96), (70, 260)]


def make(rows, d, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    x = r(rows, d) * (0.1 + torch.rand((rows, 1), generator=g) * 10) + 3 * r(rows, 1)
    return x.to(dtype), r(rows, d).to(dtype), 1.0 + 0.2 * r(d), 0.3 * r(d), r(rows, d).to(dtype), r(rows, d).to(dtype)


def parts(x, res):
    """h, h - m and r in 64 bits, and what the first two may be off by."""
    h = x.double() + (res.double() if res is not None else 0.0)
    mag = x.double().abs() + (res.double().abs() if res is not None else 0.0)
    d = h.shape[-1]
    c = h - h.mean(-1, keepdim=True)
    ec = 2 * U * mag + (d + 2) * U * mag.mean(-1, keepdim=True)
    var = c.square().mean(-1, keepdim=True)
    # a mean that is off by e adds e^2 to the mean of the squares about it, its terms 2 |c| times their own rounding
    ev = (d + 4) * U * var + ec.square().mean(-1, keepdim=True) + 2 * (c.abs() * 2 * U * (mag + c.abs())).mean(-1, keepdim=True)
    r = 1 / (var + EPS).sqrt()
    er = 0.5 * r ** 3 * ev * 1.01 + 4 * U * r
    return h, c, ec, r, er, mag


@pytest.mark.parametrize("out", ["f32", "bf16", "e4m3"])
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("rows,d", SIZES)
def test_forward(rows, d, dtype, out):
    x, res0, gamma, bias, _, _ = make(rows, d, dtype, rows + d)
    for res in (None, res0):
        for be in (bias, None):
            h, c, ec, r, er, mag = parts(x, res)
            n = c * r
            en = ec * r + c.abs() * er + U * n.abs()
            b = be.double() if be is not None else torch.zeros(d, dtype=torch.float64)
            y = n * gamma.double() + b
            ey = en * gamma.double().abs() + 2 * U * (n.abs() * gamma.double().abs() + b.abs())
            got = sdm.sdm_residual_layer_norm(x.to(DEV), gamma.to(DEV), None if be is None else be.to(DEV),
                                              None if res is None else res.to(DEV), EPS, out)
            if res is not None:
                assert got["h"].dtype == dtype
                assert ((got["h"].cpu().double() - h).abs() <= HALF[dtype] * h.abs() * (1 + 1e-6) + U * mag + 1e-38).all()
            z = got["y"].cpu().double()
            if out == "e4m3":
                s = got["scale"].cpu().double()
                assert s.shape == (rows, 1)
                want = y.abs().amax(-1, keepdim=True) / 448
                assert ((s - want).abs() <= ey.amax(-1, keepdim=True) / 448 + 2 * U * want + 1e-37).all()
                assert ((z * s - y).abs() <= 2.0 ** -4 * y.abs() * (1 + 1e-5) + 2.0 ** -10 * s + 3 * ey + 1e-37).all()
            else:
                t = {"f32": F32, "bf16": BF}[out]
                assert ((z - y).abs() <= HALF[t] * y.abs() + 1.01 * ey + 1e-37).all()


@pytest.mark.parametrize("group", [32, 128, 512])
def test_groups(group):
    for rows, d in ((3, 512), (17, 2560), (2, 8192)):
        x, res, gamma, bias, _, _ = make(rows, d, BF, group + d)
        h, c, ec, r, er, mag = parts(x, res)
        y = c * r * gamma.double() + bias.double()
        ey = (ec * r + c.abs() * er + 3 * U * (c * r).abs()) * gamma.double().abs() + 2 * U * bias.double().abs()
        got = sdm.sdm_residual_layer_norm(x.to(DEV), gamma.to(DEV), bias.to(DEV), res.to(DEV), EPS, "e4m3", group)
        s = got["scale"].cpu().double()
        assert s.shape == (rows, d // group)
        yg, eg = y.view(rows, -1, group), ey.view(rows, -1, group)
        want = yg.abs().amax(-1) / 448
        assert ((s - want).abs() <= eg.amax(-1) / 448 + 2 * U * want + 1e-37).all()
        z = got["y"].cpu().double().view(rows, -1, group) * s[..., None]
        assert ((z - yg).abs() <= 2.0 ** -4 * yg.abs() * (1 + 1e-5) + 2.0 ** -10 * s[..., None] + 3 * eg + 1e-37).all()


def test_constant_rows_and_special_values():
    """A row of one value is its bias; a NaN stays within its row; far from 0 the mean is taken off first."""
    for d in (64, 100, 1024, 3000):
        _, _, gamma, bias, _, _ = make(1, d, F32, d)
        x = torch.full((5, d), 3.0)
        x[1] = 0.0
        x[2, d // 2] = float("nan")
        x[3] = 4096.0 + (torch.arange(d) % 3)      # exact values: a variance of squares less a square would lose them
        x[4, 0] = float("inf")
        got = sdm.sdm_residual_layer_norm(x.to(DEV), gamma.to(DEV), bias.to(DEV), None, EPS, "f32")["y"].cpu()
        assert torch.equal(got[1], bias)
        e = (d + 2) * U * 3.0 / EPS ** 0.5  # the mean's rounding, over the root of eps
        assert ((got[0] - bias).abs() <= e * gamma.abs() + 2 * U * bias.abs()).all()
        assert torch.isnan(got[2]).all() and torch.isnan(got[4]).all()
        h, c, ec, r, er, mag = parts(x[3:4], None)
        want = c * r * gamma.double() + bias.double()
        assert ((got[3:4].double() - want).abs() <= (ec * r + c.abs() * er) * gamma.double().abs() + 4 * U * (want.abs() + 1)).all()


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("rows,d", SIZES + [(5000, 256), (9001, 40)])
def test_backward(rows, d, dtype):
    hb, dh, gamma, _, dy, _ = make(rows, d, dtype, 3 * rows + d)
    h, c, ec, r, er, _ = parts(hb, None)
    DY, GA = dy.double(), gamma.double()
    n, gd = c * r, GA * DY
    en = ec * r + c.abs() * er + U * n.abs()
    mean = lambda t: t.mean(-1, keepdim=True)  # noqa: E731
    want = r * (gd - mean(gd) - n * mean(gd * n))
    inner = gd.abs() + mean(gd.abs()) + n.abs() * mean((gd * n).abs())
    e = er * inner + r * ((d + 8) * U * inner + en * mean((gd * n).abs()) + n.abs() * mean(gd.abs() * en))
    per = -(-rows // 256) + 64  # rows a chain of a workgroup adds, at most
    for t in (None, dh):
        w = want if t is None else want + t.double()
        got = sdm.sdm_residual_layer_norm_backward(dy.to(DEV), hb.to(DEV), gamma.to(DEV), None if t is None else t.to(DEV), EPS)
        assert got["dx"].dtype == dtype
        mag = w.abs() + (t.double().abs() if t is not None else 0)
        assert ((got["dx"].cpu().double() - w).abs() <= 1.01 * e + 2 * U * mag + HALF[dtype] * w.abs() * 1.001 + 1e-37).all()
        dg, db = (DY * n).sum(0), DY.sum(0)
        assert ((got["dgamma"].cpu().double() - dg).abs() <= 1.01 * (DY.abs() * en).sum(0) + (per + 4) * U * (DY * n).abs().sum(0) + 1e-37).all()
        assert ((got["dbias"].cpu().double() - db).abs() <= (per + 4) * U * DY.abs().sum(0) + 1e-37).all()


def test_in_place_empty_and_refusals():
    x, res, gamma, bias, dy, dh = (t.to(DEV) for t in make(6, 96, BF, 1))
    want = sdm.sdm_residual_layer_norm(x, gamma, bias, res, EPS)
    h = res.clone()
    got = sdm.sdm_residual_layer_norm(x, gamma, bias, h, EPS, out={"h": h})
    assert got["h"] is h and torch.equal(h, want["h"]) and torch.equal(got["y"], want["y"])
    wb = sdm.sdm_residual_layer_norm_backward(dy, h, gamma, dh, EPS)
    g = dh.clone()
    gb = sdm.sdm_residual_layer_norm_backward(dy, h, gamma, g, EPS, out={"dx": g})
    assert torch.equal(g, wb["dx"]) and torch.equal(gb["dbias"], wb["dbias"])
    e = sdm.sdm_residual_layer_norm_backward(dy[:0], h[:0], gamma)
    assert (e["dgamma"] == 0).all() and (e["dbias"] == 0).all() and e["dx"].shape == (0, 96)
    assert sdm.sdm_residual_layer_norm(x[:0], gamma)["y"].shape == (0, 96)
    for bad in (lambda: sdm.sdm_residual_layer_norm(x, gamma, bias[:5]), lambda: sdm.sdm_residual_layer_norm(x, gamma, bias.to(BF)),
                lambda: sdm.sdm_residual_layer_norm(x, gamma, bias, dtype="e5m2"),
                lambda: sdm.sdm_residual_layer_norm_backward(dy, h, gamma, out={"dbeta": bias}),
                lambda: sdm.sdm_residual_layer_norm(x.t(), gamma)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(sdm.SdmError):
        sdm.sdm_residual_layer_norm(x, gamma, bias, None, EPS, "bf16", out={"y": x})


def test_gradients_against_differences():
    x, _, gamma, bias, dy, _ = (t.to(DEV) for t in make(4, 40, F32, 5))
    got = sdm.sdm_residual_layer_norm_backward(dy, x, gamma, None, EPS)
    g = torch.Generator().manual_seed(2)
    for name, grad in (("x", "dx"), ("gamma", "dgamma"), ("bias", "dbias")):
        c = {"x": x, "gamma": gamma, "bias": bias}
        v = torch.randn(c[name].shape, generator=g).to(DEV)
        s = 2.0 ** -9  # fp32 values off by some 8 half steps over it, 2.5e-4; the third derivative of rows 0.1 wide, 1e-4

        def loss(k):
            q = dict(c, **{name: c[name] + k * v})
            return float((sdm.sdm_residual_layer_norm(q["x"], q["gamma"], q["bias"], None, EPS, "f32")["y"].double() * dy.double()).sum())

        want, size = float((got[grad].double() * v.double()).sum()), float((got[grad].double() * v.double()).abs().sum())
        assert abs((loss(s) - loss(-s)) / (2 * s) - want) <= 2e-3 * size, name
