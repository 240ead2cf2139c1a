"""Residual norm and its gradients against 64 bits.

Tolerances count roundings of half a step: fp32 sums over d in some tree or
chain, at most n = d additions (2^-24 each, of sums of squares, all positive),
and a handful of products; outputs in bf16 add half a bf16 step (2^-8 relative),
e4m3 half a step of 2^-4 relative, or of its smallest number (2^-9) / 2 absolutely.
"""
import pytest
import torch

import sparse_memory_linear_amd as sdm

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
BF, F32, F8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
HALF = {BF: 2.0 ** -8, F32: 2.0 ** -24, F8: 2.0 ** -4}
EPS = 1e-6


def make(rows, d, dtype, seed, special=False):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((rows, d), generator=g) * (0.1 + torch.rand((rows, 1), generator=g) * 10)
    if special:
        x[0] = 0.0                      # a row of zeros
        if rows > 1:
            x[1] = 1e-22                # squares that underflow: eps decides
        if rows > 2:
            x[2] = 0.0
            x[2, d // 2] = 3e18         # one large value
    return x.to(dtype), torch.randn((rows, d), generator=g).to(dtype), 1.0 + 0.2 * torch.randn(d, generator=g)


def reference(x, res, gamma):
    h = x.double() + (res.double() if res is not None else 0.0)
    y = h / (h.square().mean(-1, keepdim=True) + EPS).sqrt() * gamma.double()
    return h, y


SIZES = [(1, 1), (2, 7), (5, 64), (3, 100), (8, 512), (33, 1024), (4, 1919), (3, 2048), (5, 2052), (2, 4097),
         (3, 5120), (2, 8200), (2, 8192), (1, 12001), (2, 16384), (1, 16383), (2, 6004), (1300, 96)]


@pytest.mark.parametrize("out", ["f32", "bf16", "e4m3"])
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("rows,d", SIZES)
def test_forward(rows, d, dtype, out):
    x, r, gamma = make(rows, d, dtype, rows + d)
    for res in (None, r):
        h, y = reference(x, res, gamma)
        got = sdm.sdm_residual_norm(x.to(DEV), gamma.to(DEV), None if res is None else res.to(DEV), EPS, out)
        rel = (d + 8) * 2.0 ** -24  # of y in fp32: the squares' sum, its root, three products
        hmag = x.double().abs() + (res.double().abs() if res is not None else 0.0)
        ymag = hmag / (h.square().mean(-1, keepdim=True) + EPS).sqrt() * gamma.double().abs()
        if res is not None:
            assert got["h"].dtype == dtype
            e = (got["h"].cpu().double() - h).abs()
            assert (e <= HALF[dtype] * h.abs() * (1 + 1e-6) + 2.0 ** -24 * hmag + 1e-38).all()
        z = got["y"].cpu().double()
        if out == "e4m3":
            s = got["scale"].cpu().double()
            assert s.shape == (rows, 1)
            want = y.abs().amax(-1, keepdim=True) / 448
            assert ((s - want).abs() <= (rel + 2 ** -23) * ymag.amax(-1, keepdim=True) / 448 + 1e-37).all()
            assert (z.abs() <= 448).all()
            e = (z * s - y).abs()
            # a value on a rounding border may fall to either side: half a step more than nothing, rel in all
            assert (e <= 2.0 ** -4 * y.abs() * (1 + 1e-5) + (2.0 ** -10 * s) + 3 * rel * ymag + 1e-37).all()
        else:
            t = {"f32": F32, "bf16": BF}[out]
            assert ((z - y).abs() <= HALF[t] * y.abs() + rel * ymag * (1 + 1e-3) + 1e-37).all()


@pytest.mark.parametrize("group", [32, 64, 128, 256, 512])
def test_groups(group):
    for rows, d in ((3, 512), (17, 2560), (2, 8192)):
        x, res, gamma = make(rows, d, BF, group + d, special=True)
        h, y = reference(x, res, gamma)
        got = sdm.sdm_residual_norm(x.to(DEV), gamma.to(DEV), res.to(DEV), EPS, "e4m3", group)
        yg = y.view(rows, -1, group)
        s = got["scale"].cpu().double()
        assert s.shape == (rows, d // group)
        rel = (d + 8) * 2.0 ** -24
        mag = (x.double().abs() + res.double().abs()) / (h.square().mean(-1, keepdim=True) + EPS).sqrt() * gamma.double().abs()
        mg = mag.view(rows, -1, group)
        assert ((s - yg.abs().amax(-1) / 448).abs() <= (rel + 2 ** -23) * mg.amax(-1) / 448 + 1e-37).all()
        z = got["y"].cpu().double().view(rows, -1, group) * s[..., None]
        assert ((z - yg).abs() <= 2.0 ** -4 * yg.abs() * (1 + 1e-5) + 2.0 ** -10 * s[..., None] + 3 * rel * mg + 1e-37).all()


def test_rows_of_zeros_and_extremes():
    for d in (64, 1024, 2999):
        x, _, gamma = make(4, d, F32, d, special=True)
        h, y = reference(x, None, gamma)
        got = sdm.sdm_residual_norm(x.to(DEV), gamma.to(DEV), None, EPS, "f32")["y"].cpu().double()
        assert (got[0] == 0).all() and torch.isfinite(got).all()
        assert ((got - y).abs() <= (d + 8) * 2.0 ** -24 * y.abs() + 1e-37).all()
        q = sdm.sdm_residual_norm(x.to(DEV), gamma.to(DEV), None, EPS, "e4m3")
        assert q["scale"][0] == 0 and (q["y"][0].float() == 0).all()
        x[3, 5] = float("nan")  # a NaN stays within its row
        got = sdm.sdm_residual_norm(x.to(DEV), gamma.to(DEV), None, EPS, "e4m3")
        assert torch.isnan(got["y"][3].float()).all() and torch.isfinite(got["y"][:3].float()).all()


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("rows,d", SIZES + [(5000, 256), (9001, 40)])
def test_backward(rows, d, dtype):
    h, dy, gamma = make(rows, d, dtype, 3 * rows + d)
    g = torch.Generator().manual_seed(1)
    dh = torch.randn((rows, d), generator=g).to(dtype)
    H, DY, GA = h.double(), dy.double(), gamma.double()
    r = 1 / (H.square().mean(-1, keepdim=True) + EPS).sqrt()
    n = H * r
    want = r * (GA * DY - n * (GA * DY * n).mean(-1, keepdim=True))
    dgamma = (DY * n).sum(0)
    rel = (3 * d + 16) * 2.0 ** -24
    mag = r * ((GA * DY).abs() + n.abs() * (GA * DY * n).abs().mean(-1, keepdim=True))
    for t in (None, dh):
        w = want if t is None else want + t.double()
        got = sdm.sdm_residual_norm_backward(dy.to(DEV), h.to(DEV), gamma.to(DEV), None if t is None else t.to(DEV), EPS)
        assert got["dx"].dtype == dtype
        m = mag if t is None else mag + t.double().abs()
        assert ((got["dx"].cpu().double() - w).abs() <= HALF[dtype] * w.abs() + rel * m + 1e-37).all()
        # per row a normalised value's error, and the sum over the rows
        tol = (rows + d + 16) * 2.0 ** -24 * (DY * n).abs().sum(0)
        assert ((got["dgamma"].cpu().double() - dgamma).abs() <= tol + 1e-37).all()


def test_gradient_against_differences():
    x, dy, gamma = make(6, 50, F32, 4)
    got = sdm.sdm_residual_norm_backward(dy.to(DEV), x.to(DEV), gamma.to(DEV), None, EPS)
    g = torch.Generator().manual_seed(3)
    d, e = torch.randn(x.shape, generator=g, dtype=torch.float64), torch.randn(50, generator=g, dtype=torch.float64)
    f = lambda s: (reference(x.double() + s * d, None, gamma.double() + s * e)[1] * dy.double()).sum()  # noqa: E731
    s = 2.0 ** -18
    want = (f(s) - f(-s)) / (2 * s)
    a, b = got["dx"].cpu().double() * d, got["dgamma"].cpu().double() * e
    assert abs(want - (a.sum() + b.sum())) <= 1e-5 * (a.abs().sum() + b.abs().sum())


def test_in_place_mixed_types_and_shapes():
    x, res, gamma = (t.to(DEV) for t in make(12, 256, BF, 9))
    resf = res.float()
    x3 = x.view(3, 4, 256)
    a = sdm.sdm_residual_norm(x3, gamma, resf.view(3, 4, 256), EPS, "e4m3", 64)
    assert a["h"].dtype == F32 and a["scale"].shape == (3, 4, 4) and a["y"].shape == (3, 4, 256)
    b = sdm.sdm_residual_norm(x, gamma, resf.clone(), EPS, "e4m3", 64)
    assert torch.equal(a["h"].view(12, 256), b["h"]) and torch.equal(a["y"].view(12, 256).view(torch.uint8), b["y"].view(torch.uint8))
    r2 = resf.clone()
    c = sdm.sdm_residual_norm(x, gamma, r2, EPS, "e4m3", 64, out={"h": r2})
    assert c["h"].data_ptr() == r2.data_ptr() and torch.equal(r2, b["h"])
    # gradients in fp32 for a bf16 stream, written over dh
    dy = torch.randn(12, 256, device=DEV)
    dh = torch.randn(12, 256, device=DEV)
    u = sdm.sdm_residual_norm_backward(dy, x, gamma, dh, EPS)
    d2 = dh.clone()
    v = sdm.sdm_residual_norm_backward(dy, x, gamma, d2, EPS, out={"dx": d2})
    assert torch.equal(u["dx"], d2) and torch.equal(u["dgamma"], v["dgamma"])


def test_h_over_x_and_all_type_pairs():
    for xt in (BF, F32):
        for ht in (BF, F32):
            x, r, gamma = make(7, 300, F32, 12)
            x, r, gamma = x.to(xt).to(DEV), r.to(ht).to(DEV), gamma.to(DEV)
            a = sdm.sdm_residual_norm(x, gamma, r, EPS, "f32")
            h, y = reference(x.cpu(), r.cpu(), gamma.cpu())
            mag = (x.double().abs() + r.double().abs()).cpu()
            assert ((a["h"].cpu().double() - h).abs() <= HALF[ht] * h.abs() * (1 + 1e-6) + 2.0 ** -24 * mag).all()
            ymag = mag / (h.square().mean(-1, keepdim=True) + EPS).sqrt() * gamma.cpu().double().abs()
            assert ((a["y"].cpu().double() - y).abs() <= 308 * 2.0 ** -24 * ymag * (1 + 1e-3)).all()
            if xt == ht:
                x2 = x.clone()
                b = sdm.sdm_residual_norm(x2, gamma, r, EPS, "f32", out={"h": x2})
                assert b["h"].data_ptr() == x2.data_ptr() and torch.equal(x2, a["h"]) and torch.equal(a["y"], b["y"])
            # gradients of either type over a stream of either type
            dy = torch.randn(7, 300, device=DEV).to(xt)
            g = sdm.sdm_residual_norm_backward(dy, a["h"], gamma, None, EPS)
            H, DY, GA = a["h"].cpu().double(), dy.cpu().double(), gamma.cpu().double()
            rr = 1 / (H.square().mean(-1, keepdim=True) + EPS).sqrt()
            n = H * rr
            w = rr * (GA * DY - n * (GA * DY * n).mean(-1, keepdim=True))
            m = rr * ((GA * DY).abs() + n.abs() * (GA * DY * n).abs().mean(-1, keepdim=True))
            assert g["dx"].dtype == xt
            assert ((g["dx"].cpu().double() - w).abs() <= HALF[xt] * w.abs() + 916 * 2.0 ** -24 * m).all()


def test_offsets_beyond_32_bits():
    rows, d = 2_200_003, 1024
    x = torch.empty((rows, d), dtype=BF, device=DEV).normal_()
    gamma = torch.ones(d, device=DEV)
    a = sdm.sdm_residual_norm(x, gamma, None, EPS, "e4m3", 128)
    b = sdm.sdm_residual_norm(x[-9:].clone(), gamma, None, EPS, "e4m3", 128)
    assert torch.equal(a["y"][-9:].view(torch.uint8), b["y"].view(torch.uint8)) and torch.equal(a["scale"][-9:], b["scale"])
    g = sdm.sdm_residual_norm_backward(x, x, gamma, x)
    h = sdm.sdm_residual_norm_backward(x[-9:].clone(), x[-9:].clone(), gamma, x[-9:].clone())
    assert torch.equal(g["dx"][-9:], h["dx"])


def test_more_rows_than_one_side_of_a_grid():
    rows = (1 << 28) + 37
    x = torch.full((rows, 1), -3.0, dtype=BF, device=DEV)
    x[1 << 28:] = 5.0
    y = sdm.sdm_residual_norm(x, torch.full((1,), 2.0, device=DEV), None, 0.0)["y"]
    assert (y[:1 << 28] == -2.0).all() and (y[1 << 28:] == 2.0).all()  # h / |h| gamma


def test_no_rows():
    x = torch.empty((0, 64), dtype=BF, device=DEV)
    gamma = torch.ones(64, device=DEV)
    assert sdm.sdm_residual_norm(x, gamma, x, EPS, "e4m3")["y"].shape == (0, 64)
    got = sdm.sdm_residual_norm_backward(x, x, gamma)
    assert (got["dgamma"] == 0).all() and got["dx"].shape == (0, 64)


def test_captured_and_replayed():
    x, res, gamma = (t.to(DEV) for t in make(700, 1024, BF, 2))
    run = lambda: {**sdm.sdm_residual_norm(x, gamma, res, EPS, "e4m3", 128), **sdm.sdm_residual_norm_backward(res, x, gamma)}  # noqa: E731
    want = run()
    s, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        run()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=s):
            got = run()
    for _ in range(3):
        for t in got.values():
            t.view(torch.uint8).fill_(1)
        graph.replay()
        torch.cuda.synchronize()
        for name in want:
            assert torch.equal(got[name].view(torch.uint8), want[name].view(torch.uint8)), name


def test_refusals():
    x, res, gamma = (t.to(DEV) for t in make(4, 96, BF, 1))
    for call in (lambda: sdm.sdm_residual_norm(x, gamma[:-1].contiguous()), lambda: sdm.sdm_residual_norm(x, gamma.to(BF)),
                 lambda: sdm.sdm_residual_norm(x, gamma, res[:2]), lambda: sdm.sdm_residual_norm(x, gamma, dtype="f16"),
                 lambda: sdm.sdm_residual_norm(x.half(), gamma), lambda: sdm.sdm_residual_norm(x.t(), gamma),
                 lambda: sdm.sdm_residual_norm(x, gamma, dtype="e4m3", group=64),
                 lambda: sdm.sdm_residual_norm(x, gamma, out={"h": res}),
                 lambda: sdm.sdm_residual_norm_backward(x, res, gamma, res.float()),
                 lambda: sdm.sdm_residual_norm_backward(x, res[:2], gamma)):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: sdm.sdm_residual_norm(x, gamma, dtype="e4m3", group=48), lambda: sdm.sdm_residual_norm(x, gamma, eps=-1.0),
                 lambda: sdm.sdm_residual_norm(x, gamma, dtype="bf16", group=32),
                 lambda: sdm.sdm_residual_norm(x, gamma, out={"y": x}),
                 lambda: sdm.sdm_residual_norm(torch.zeros(1, 16400, device=DEV), torch.zeros(16400, device=DEV))):
        with pytest.raises(sdm.SdmError):
            call()


@pytest.mark.parametrize("group", [0, 32, 128, 512])
def test_codes_are_the_rounded_quotients(group):
    """The fp32 output holds the y that the 8-bit one is made of: its scale is the fp32 quotient
    max |y| / 448 (at least 2^-126) and its codes the fp32 quotients y / scale, to nearest even, bit
    for bit; also for rows so small that eps decides and y / scale passes through denormal numbers."""
    for rows, d in ((700, 1024), (9, 8192), (3, 512)) + (((400, 1919), (5000, 40)) if group == 0 else ()):
        for size in (1.0, 1e-30, 1e-35, 1e-39):
            x, res, gamma = make(rows, d, F32 if size < 1 else BF, group + rows)
            x, res, gamma = (x * size).to(DEV), (res * size).to(DEV), gamma.to(DEV)
            y = sdm.sdm_residual_norm(x, gamma, res, EPS, "f32")["y"].cpu().view(rows, -1, group or d)
            got = sdm.sdm_residual_norm(x, gamma, res, EPS, "e4m3", group)
            scale = (y.abs().amax(-1) / 448.0).clamp_min(2.0 ** -126)
            assert torch.equal(got["scale"].cpu(), scale)
            codes = (y / scale[..., None]).to(F8).view(rows, d)
            assert torch.equal(got["y"].cpu().view(torch.uint8), codes.view(torch.uint8))


@pytest.mark.parametrize("d", [512, 1919, 8192])
def test_scales_of_rows_that_are_not_finite(d):
    """A scale is 0 only over zeros: over a NaN, or an infinity (whose y, infinity / infinity, is one), it is a NaN."""
    x, _, gamma = make(6, d, F32, d)
    x[1, 7], x[2, d - 1], x[3, 300], x[4] = float("nan"), float("inf"), -float("inf"), 0.0
    for group in (0,) if d % 128 else (0, 128):
        n = d // (group or d)
        got = sdm.sdm_residual_norm(x.to(DEV), gamma.to(DEV), None, EPS, "e4m3", group)
        s, y = got["scale"].cpu(), got["y"].cpu().float().view(6, n, -1)
        want = torch.zeros(6, n, dtype=torch.bool)
        want[1] = True                                       # the norm of a row with a NaN is one
        want[2, -1] = want[3, 300 // (group or d)] = True    # beside an infinity all else is 0
        assert torch.equal(torch.isnan(s), want) and torch.equal(torch.isnan(y).all(-1), want)
        assert torch.equal(torch.isnan(y).any(-1), want)
        s[want], y[want] = 0.0, 0.0
        assert (s[1:5] == 0).all() and (y[1:5] == 0).all() and (s[0] > 0).all() and (s[5] > 0).all()
        g = gamma.clone()
        g[5] = float("nan")                                  # and so is that of a column
        s = sdm.sdm_residual_norm(x[:1].to(DEV), g.to(DEV), None, EPS, "e4m3", group)["scale"].cpu()
        assert torch.isnan(s[0, 0]) and (s[0, 1:] > 0).all()


# Rows in turn: 9001 x 512 and below take 16 to 64 threads a row (4 to 16 rows a workgroup, 1024
# workgroups), 1536 to 4096 columns 256 threads, more 1024 threads (256 workgroups).
LOOPS = [(40000, 40, 16, 1024), (20000, 200, 8, 1024), (9001, 512, 4, 1024), (9001, 1001, 4, 1024), (2600, 1536, 1, 1024),
         (2600, 3001, 1, 1024), (700, 8192, 1, 256), (700, 12001, 1, 256)]


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("rows,d,together,blocks", LOOPS)
def test_backward_of_several_rows_a_thread_group(rows, d, together, blocks, dtype):
    """dgamma's sums are chains of a thread group's rows, of a workgroup's groups, of 1 in 64 workgroups,
    and 6 levels of pairs: a rounding of each is of at most the sum of the magnitudes."""
    h, dy, gamma = make(rows, d, dtype, rows + 5 * d)
    H, DY, GA = h.double(), dy.double(), gamma.double()
    r = 1 / (H.square().mean(-1, keepdim=True) + EPS).sqrt()
    n = H * r
    want = r * (GA * DY - n * (GA * DY * n).mean(-1, keepdim=True))
    mag = r * ((GA * DY).abs() + n.abs() * (GA * DY * n).abs().mean(-1, keepdim=True))
    got = sdm.sdm_residual_norm_backward(dy.to(DEV), h.to(DEV), gamma.to(DEV), None, EPS)
    assert ((got["dx"].cpu().double() - want).abs() <= HALF[dtype] * want.abs() + (3 * d + 16) * 2.0 ** -24 * mag + 1e-37).all()
    # the squares' sum of a row: a thread's pieces of 8, 10 levels over its threads; half of that in its root
    own = 8 + 10 + 6
    chain = (rows + together * blocks - 1) // (together * blocks) + together + (blocks + 63) // 64 + 6
    tol = (own + chain) * 2.0 ** -24 * (DY * n).abs().sum(0)
    assert ((got["dgamma"].cpu().double() - (DY * n).sum(0)).abs() <= tol + 1e-37).all()


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("rows,d", [c[:2] for c in LOOPS] + [(9001, 40), (5000, 256), (1500, 1024)])
def test_no_row_is_lost_or_added_twice(rows, d, dtype):
    """Rows of +-1 without eps have a norm of 1, and whole gradients: dgamma is a sum of whole numbers below 2^24, and exact."""
    g = torch.Generator().manual_seed(rows)
    h = torch.randint(0, 2, (rows, d), generator=g).mul_(2).sub_(1).to(dtype)
    dy = torch.randint(-9, 10, (rows, d), generator=g).to(dtype)
    got = sdm.sdm_residual_norm_backward(dy.to(DEV), h.to(DEV), torch.ones(d, device=DEV), None, 0.0)
    assert torch.equal(got["dgamma"].cpu().double(), (dy.double() * h.double()).sum(0))


@pytest.mark.parametrize("rows,d", [(5, 300), (7, 1024), (2600, 1536), (700, 8200)])
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_dx_over_dy_and_over_h(rows, d, dtype):
    h, dy, gamma = (t.to(DEV) for t in make(rows, d, dtype, d))
    dh = torch.flip(dy, (0, 1)).contiguous()
    for behind in (None, dh):
        want = sdm.sdm_residual_norm_backward(dy, h, gamma, behind, EPS)
        for over in ("dy", "h") + (("dh",) if behind is not None else ()):
            a = {"dy": dy.clone(), "h": h.clone(), "dh": None if behind is None else behind.clone()}
            got = sdm.sdm_residual_norm_backward(a["dy"], a["h"], gamma, a["dh"], EPS, out={"dx": a[over]})
            assert got["dx"].data_ptr() == a[over].data_ptr()
            assert torch.equal(got["dx"], want["dx"]) and torch.equal(got["dgamma"], want["dgamma"]), over


def test_gradient_of_a_bf16_stream():
    """The norm is that of the fp32 sum, its gradient's that of the stored one, half a bf16 step (2^-8) off an
    element: n is off by 2^-8 |n| from that and, through r, by at most as much again, so dx in fp32 is by 2 * 2^-8
    times each of r's three uses in its terms, 6 * 2^-8 of their magnitudes (dgamma: 2 * 2^-8), and a little in second order."""
    x, res, gamma = make(50, 1000, BF, 21)
    dy = torch.randn((50, 1000), generator=torch.Generator().manual_seed(8))
    X, R, GA = (t.double().requires_grad_() for t in (x, res, gamma))
    y = reference(X, R, GA)[1]
    dx, _, dgamma = torch.autograd.grad((y * dy.double()).sum(), [X, R, GA])
    f = sdm.sdm_residual_norm(x.to(DEV), gamma.to(DEV), res.to(DEV), EPS, "bf16")
    got = sdm.sdm_residual_norm_backward(dy.to(DEV), f["h"], gamma.to(DEV), None, EPS)
    h = x.double() + res.double()
    r = 1 / (h.square().mean(-1, keepdim=True) + EPS).sqrt()
    n, gd = (h * r).abs(), (gamma * dy).double().abs()
    mag = r * (gd + n * (gd * n).mean(-1, keepdim=True))
    assert ((got["dx"].cpu().double() - dx).abs() <= 6.1 * 2.0 ** -8 * mag).all()
    assert ((got["dgamma"].cpu().double() - dgamma).abs() <= 2.1 * 2.0 ** -8 * (n * dy.double().abs()).sum(0)).all()
