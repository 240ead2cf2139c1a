"""Slot counts, balance loss and its gradient against 64 bits.

Counts are whole numbers and equal. A weight is added to 2^-s, s >= 40 for calls
of up to 2^21 selections, so a mass is off by at most its selections times 2^-41
and half an fp32 step; the loss and dwt are formed in 64 bits from those and
rounded once more (dwt by one more product).
"""
import pytest
import torch

import sparse_memory_linear_amd as sdm
from sparse_memory_linear_amd import inputs

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


def make(B, H, T, K, N, seed, mask="none", skew=2.0):
    g = torch.Generator().manual_seed(seed)
    idx = (N * torch.rand((B, H, T, K), generator=g) ** skew).to(torch.int32).clamp_(0, N - 1)
    wt = torch.softmax(torch.randn((B, H, T, K), generator=g) * 2, -1)
    m = None
    if mask == "some":
        m = (torch.rand((B, T), generator=g) < 0.6).to(torch.uint8) * 3
    elif mask == "empty":
        m = torch.zeros((B, T), dtype=torch.bool)
    return idx, wt, m


def reference(idx, wt, N, mask):
    B, H, T, K = idx.shape
    keep = torch.ones(B, T, dtype=torch.bool) if mask is None else mask != 0
    n = int(keep.sum())
    ok = keep[:, None, :, None] & (idx >= 0) & (idx < N)
    counts, mass = torch.zeros(H, N, dtype=torch.int64), torch.zeros(H, N, dtype=torch.float64)
    for h in range(H):
        at = idx[:, h][ok[:, h]].long()
        counts[h] = torch.bincount(at, minlength=N)
        mass[h] = torch.bincount(at, weights=wt[:, h][ok[:, h]].double(), minlength=N)
    loss = N * (counts.double() * mass).sum(-1) / max(n * K, 1) / max(n, 1)
    dwt = torch.zeros(idx.shape, dtype=torch.float64)
    if n:
        f = counts.double() / (n * K)
        for h in range(H):
            dwt[:, h] = torch.where(ok[:, h], N / n * f[h][idx[:, h].long().clamp(0, N - 1)], 0.0)
    return counts, mass, n, loss, dwt


def check(idx, wt, N, mask, dloss):
    counts, mass, n, loss, dwt = reference(idx, wt, N, mask)
    D = lambda t: None if t is None else t.to(DEV)  # noqa: E731
    got = sdm.sdm_balance_forward(D(idx), D(wt), N, D(mask))
    assert torch.equal(got["counts"].cpu().long(), counts)
    assert int(got["tokens"]) == n
    e = (got["mass"].cpu().double() - mass).abs()
    assert (e <= 2.0 ** -24 * mass.abs() + counts * 2.0 ** -41).all()
    # N sum count * mass off by N sum count^2 2^-41 at most
    slack = N * (counts.double() ** 2).sum(-1) / max(n, 1) ** 2 / idx.shape[3] * 2.0 ** -41
    assert ((got["loss"].cpu().double() - loss).abs() <= 2.0 ** -24 * loss.abs() * 1.01 + slack).all()
    d = sdm.sdm_balance_backward(D(idx), got["counts"], got["tokens"], D(dloss), D(mask)).cpu().double()
    want = dwt * dloss.double()[None, :, None, None]
    assert ((d - want).abs() <= 3 * 2.0 ** -24 * want.abs()).all()
    assert (d[want == 0] == 0).all()
    return got


SIZES = [(1, 1, 1, 1, 1), (1, 1, 1, 8, 16), (2, 3, 7, 5, 49), (1, 2, 300, 64, 4096), (3, 1, 1000, 8, 262144),
         (2, 8, 129, 33, 65536), (1, 4, 64, 256, 256), (5, 5, 11, 3, 10007), (2, 2, 2500, 64, 65536)]


@pytest.mark.parametrize("mask", ["none", "some", "empty"])
@pytest.mark.parametrize("B,H,T,K,N", SIZES)
def test_counts_loss_and_gradient(B, H, T, K, N, mask):
    idx, wt, m = make(B, H, T, K, N, B + T + K + N, mask)
    check(idx, wt, N, m, 0.5 + torch.arange(H, dtype=torch.float32))


def test_one_slot_takes_everything_and_even_use():
    idx = torch.full((2, 2, 3000, 4), 17, dtype=torch.int32)
    wt = torch.full((2, 2, 3000, 4), 0.25)
    got = check(idx, wt, 64, None, torch.ones(2))
    assert got["counts"][0, 17] == 2 * 3000 * 4 and got["loss"][0] == 64.0
    even = torch.arange(64, dtype=torch.int32).view(1, 1, 16, 4)
    assert check(even, torch.full((1, 1, 16, 4), 0.25), 64, None, torch.ones(1))["loss"][0] == 1.0


def test_counts_beyond_16_bits_and_the_largest_table():
    idx = torch.full((2, 2, 9000, 8), 17, dtype=torch.int32)
    idx[0, 0, :, 0] = 3
    got = check(idx, torch.full((2, 2, 9000, 8), 0.125), 64, None, torch.ones(2))
    assert got["counts"][0, 17] == 2 * 9000 * 8 - 9000
    idx, wt, m = make(1, 16, 10300, 64, 81920, 9, "some")  # 81920 counts of 16 bits: all of a CU's LDS
    check(idx, wt, 81920, m, torch.ones(16))
    idx, wt, m = make(1, 16, 10300, 64, 81921, 9)
    check(idx, wt, 81921, None, torch.ones(16))


def test_selections_out_of_range_are_left_out():
    idx, wt, m = make(2, 2, 50, 8, 100, 3, "some")
    idx[0, 0, :, 0] = 100
    idx[1, 1, :, 3] = -1
    idx[0, 1, 5, 2] = 2 ** 31 - 1
    check(idx, wt, 100, m, torch.tensor([2.0, -1.0]))


def test_values_at_masked_tokens_and_beyond_the_range():
    idx, wt, m = make(2, 3, 40, 8, 64, 4, "some")
    off = (m == 0)[:, None, :, None].expand_as(wt)
    wt[off] = float("nan")
    idx[off] = -5
    clean = wt.clone()
    got = check(idx, clean.nan_to_num(0.0), 64, m, torch.ones(3))
    got2 = sdm.sdm_balance_forward(idx.to(DEV), wt.to(DEV), 64, m.to(DEV))
    for name in got:
        assert torch.equal(got[name], got2[name]), name
    b, t = (m != 0).nonzero()[0].tolist()
    for v in (float("nan"), float("inf"), -3.0):
        wt[b, 1, t, 2] = v
        bad = sdm.sdm_balance_forward(idx.to(DEV), wt.to(DEV), 64, m.to(DEV))
        assert torch.isnan(bad["loss"][1]) and torch.isnan(bad["mass"][1]).all()
        assert torch.equal(bad["loss"][::2], got["loss"][::2]) and torch.equal(bad["counts"], got["counts"])


def test_many_selections_repeat_bit_for_bit():
    idx, wt, _ = make(2, 2, 9000, 64, 4096, 8)
    a = check(idx, wt, 4096, None, torch.ones(2))
    for _ in range(3):
        b = sdm.sdm_balance_forward(idx.to(DEV), wt.to(DEV), 4096)
        for name in a:
            assert torch.equal(a[name], b[name]), name


def test_offsets_beyond_32_bits():
    """2.3 G selections in all (17 heads): the last head as a call of its own."""
    H, T, K, N = 17, 2_100_000, 64, 4096
    idx = torch.empty((1, H, T, K), dtype=torch.int32, device=DEV).random_(0, N)
    wt = torch.empty((1, H, T, K), device=DEV).fill_(1 / 64)
    dl = torch.ones(H, device=DEV)
    a = sdm.sdm_balance_forward(idx, wt, N)
    d = sdm.sdm_balance_backward(idx, a["counts"], a["tokens"], dl)
    i, w = idx[:, -1:].clone(), wt[:, -1:].clone()
    b = sdm.sdm_balance_forward(i, w, N)
    assert torch.equal(a["counts"][-1:], b["counts"]) and torch.equal(a["mass"][-1:], b["mass"])
    assert (a["counts"].sum(-1) == T * K).all() and torch.equal(a["loss"][-1:], b["loss"])
    assert torch.equal(d[:, -1:], sdm.sdm_balance_backward(i, b["counts"], b["tokens"], dl[:1]))


def test_one_sequence_of_more_than_2_to_24_masked_tokens():
    T, N = (1 << 24) + 5001, 1 << 18
    mask = (torch.arange(T, device=DEV) % 7 < 3).to(torch.uint8)[None]
    mask[0, 1 << 24:] = 1 - mask[0, 1 << 24:]
    keep = mask[0] != 0
    # 13 heads of 20 ranges: a workgroup walks the whole sequence
    idx = torch.randint(0, N, (1, 13, T, 1), device=DEV, dtype=torch.int32)
    wt = torch.ones((1, 13, T, 1), device=DEV)
    got = sdm.sdm_balance_forward(idx, wt, N, mask)
    assert int(got["tokens"]) == int(keep.sum())
    for h in (0, 12):
        want = torch.bincount(idx[0, h, keep, 0], minlength=N)
        assert torch.equal(got["counts"][h].long(), want)
        assert torch.equal(got["mass"][h], want.float())  # whole numbers below 2^24
    del idx, wt, got
    # 129 heads of 16 slots: so does the gradient's, with its counts in LDS
    idx = torch.zeros((1, 129, T, 1), device=DEV, dtype=torch.int32)
    n = int(keep.sum())
    counts = torch.full((129, 16), n, device=DEV, dtype=torch.int32)
    d = sdm.sdm_balance_backward(idx, counts, torch.tensor([n], device=DEV, dtype=torch.int32),
                                 torch.ones(129, device=DEV), mask)
    assert torch.equal((d != 0)[0, :, :, 0], keep[None].expand(129, T))


def test_no_tokens():
    z = sdm.sdm_balance_forward(torch.empty((0, 2, 5, 4), dtype=torch.int32, device=DEV), torch.empty((0, 2, 5, 4), device=DEV), 9)
    assert (z["counts"] == 0).all() and (z["mass"] == 0).all() and (z["loss"] == 0).all() and int(z["tokens"]) == 0


def test_gradient_against_differences():
    """The loss is linear in the weights at fixed slots, so one difference in 64 bits is the gradient."""
    idx, wt, m = make(2, 2, 30, 4, 36, 6, "some")
    g = torch.Generator().manual_seed(1)
    d = torch.randn(wt.shape, generator=g, dtype=torch.float64)
    dl = torch.tensor([0.3, 2.0])
    loss = lambda w: (reference(idx, w, 36, m)[3] * dl.double()).sum()  # noqa: E731
    want = loss(wt.double() + d) - loss(wt.double())
    got = sdm.sdm_balance_forward(idx.to(DEV), wt.to(DEV), 36, m.to(DEV))
    grad = sdm.sdm_balance_backward(idx.to(DEV), got["counts"], got["tokens"], dl.to(DEV), m.to(DEV)).cpu().double()
    assert abs(want - (grad * d).sum()) <= 1e-6 * (grad * d).abs().sum()


def test_on_an_addressing_result_and_captured():
    wl = inputs.get("small", T=512)
    x = {k: v.to(DEV) for k, v in inputs.make_inputs(wl).items()}
    idx, wt, _, _ = sdm.sdm_address(x["q_w"], x["q_r"], x["subkeys"], x["subkeys"], wl.W, wl.R)
    dl = torch.ones(wl.H, device=DEV)

    def run():
        o = sdm.sdm_balance_forward(idx, wt, wl.N)
        o["dwt"] = sdm.sdm_balance_backward(idx, o["counts"], o["tokens"], dl)
        return o
    check(idx.cpu(), wt.cpu(), wl.N, None, dl.cpu())
    want = run()
    s, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        run()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=s):
            got = run()
    for _ in range(4):
        for t in got.values():
            t.fill_(3)
        run()
        graph.replay()
        torch.cuda.synchronize()
        for name in want:
            assert torch.equal(got[name], want[name]), name


def test_refusals():
    idx, wt, _ = make(2, 2, 5, 4, 16, 1)
    idx, wt = idx.to(DEV), wt.to(DEV)
    m = torch.ones((2, 5), dtype=torch.uint8, device=DEV)
    for call in (lambda: sdm.sdm_balance_forward(idx.long(), wt, 16), lambda: sdm.sdm_balance_forward(idx, wt[:1], 16),
                 lambda: sdm.sdm_balance_forward(idx, wt, 16, m[:1]), lambda: sdm.sdm_balance_forward(idx, wt, 16, m.float()),
                 lambda: sdm.sdm_balance_forward(idx, wt, 0), lambda: sdm.sdm_balance_forward(idx, wt, (1 << 18) + 1)):
        with pytest.raises(ValueError):
            call()
    got = sdm.sdm_balance_forward(idx, wt, 16, m)
    with pytest.raises(ValueError):
        sdm.sdm_balance_backward(idx, got["counts"][:1].contiguous(), got["tokens"], torch.ones(2, device=DEV))
    with pytest.raises(sdm.SdmError):
        sdm.sdm_balance_forward(idx, wt, 16, workspace=torch.empty(16, dtype=torch.uint8, device=DEV))


def test_no_heads():
    """No head, no selection: nothing is counted, so no token either."""
    used = torch.full((1,), 7, dtype=torch.int32, device=DEV)
    z = sdm.sdm_balance_forward(torch.empty((2, 0, 5, 4), dtype=torch.int32, device=DEV), torch.empty((2, 0, 5, 4), device=DEV), 9,
                                out={"tokens": used})
    assert z["counts"].shape == (0, 9) and z["loss"].shape == (0,) and int(z["tokens"]) == 0
