"""Adapters with an fp32 output: what lies between the two products is held in fp32
too, however many rows the batch has.

Tolerances.  u = 2^-24.  One product of each kind alone (one element of x that is
not zero, and one of a row of b): a x is exact, its product with the scale rounds
once, three bf16 terms hold that exactly, their products with b are exact, up to
three matrix instructions add them within 1.5 ulps, 3 u, each, and base is added
with one rounding more: 11 u of the value and u of what base adds.  Dense inputs:
with M the magnitudes that the two products add, the first is off by (8 + 1.5 k /
32) 2 u M, the second, with three terms, by (8 + 4.5 rank / 32) 2 u M, and scale,
parts and base add 20 roundings.
"""

import numpy as np
import pytest
import torch

import block_scaled_mxfp4_amd as B

pytestmark = pytest.mark.gpu

BF, F32, D = torch.bfloat16, torch.float32, torch.float64
U = 2.0 ** -24
RANKS = [8, 16, 24, 32, 64, 72, 128, 256]                # every kernel of the second product, and ranks between
BATCHES = {"one_launch": [1] * 40, "tiles_of_one": [30, 0, 45], "tiles_of_four": [1] * 140 + [60],
           "tiles_of_sixteen": [700, 3, 0, 1, 90]}


def setup(batch, rank, seed):
    counts = BATCHES[batch]
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    rng = np.random.RandomState(seed)
    offsets = torch.tensor([0] + list(np.cumsum(counts)), dtype=torch.int32, device="cuda")
    adapter = torch.from_numpy(rng.randint(-1, 3, len(counts)).astype(np.int32)).cuda()
    adapter[0] = 1
    of_row = torch.repeat_interleave(adapter.long(), offsets.diff().long())
    scales = 0.5 + torch.rand(3, generator=g, device="cuda")
    return g, sum(counts), offsets, adapter, of_row, scales


@pytest.mark.parametrize("rank", RANKS)
@pytest.mark.parametrize("batch", list(BATCHES))
def test_one_product_each(batch, rank):
    g, rows, offsets, adapter, of_row, scales = setup(batch, rank, rank)
    k, n = 72, 136
    at = torch.randint(0, k, (rows,), generator=g, device="cuda")
    x = torch.zeros(rows, k, dtype=BF, device="cuda")
    x[torch.arange(rows, device="cuda"), at] = torch.randn(rows, generator=g, device="cuda").to(BF)
    a = torch.randn(3, rank, k, generator=g, device="cuda").to(BF)
    b = torch.zeros(3, n, rank, dtype=BF, device="cuda")
    place = torch.randint(0, rank, (3, n), generator=g, device="cuda")
    b.scatter_(2, place[..., None], torch.randn(3, n, 1, generator=g, device="cuda").to(BF))
    on = of_row >= 0
    i = of_row.clamp(min=0)
    t = scales.to(D)[i, None] * (a.to(D)[i, :, at] * x.to(D)[torch.arange(rows, device="cuda"), at][:, None])
    delta = t.gather(1, place[i]) * b.to(D)[i].gather(2, place[i][..., None])[..., 0] * on[:, None]
    for base in (None, torch.randn(rows, n, generator=g, device="cuda")):
        got = B.situ_moe_adapters(x, a, b, offsets, adapter, base=base, scales=scales, out_dtype=F32)
        want = delta if base is None else delta + base.to(D)
        tol = 11 * U * delta.abs() + (0.0 if base is None else U * (want.abs() + 11 * U * delta.abs()))
        bad = ~((got.to(D) - want).abs() <= tol)
        assert not bad.any(), (int(bad.sum()), bad.nonzero()[0].tolist(), got[bad][0].item(), want[bad][0].item())


@pytest.mark.parametrize("rank", RANKS)
@pytest.mark.parametrize("batch", list(BATCHES))
def test_dense(batch, rank):
    g, rows, offsets, adapter, of_row, scales = setup(batch, rank, 100 + rank)
    k, n = 200, 264
    x = torch.randn(rows, k, generator=g, device="cuda").to(BF)
    a = (k ** -0.5 * torch.randn(3, rank, k, generator=g, device="cuda")).to(BF)
    b = (rank ** -0.5 * torch.randn(3, n, rank, generator=g, device="cuda")).to(BF)
    base = torch.randn(rows, n, generator=g, device="cuda")
    want, mag = base.to(D), torch.zeros(rows, n, dtype=D, device="cuda")
    for i in range(3):
        on = of_row == i
        c, xs, aa, bb = scales[i].to(D), x[on].to(D), a[i].to(D), b[i].to(D)
        want[on] += c * (xs @ aa.t()) @ bb.t()
        mag[on] = c * (xs.abs() @ aa.abs().t()) @ bb.abs().t()
    got = B.situ_moe_adapters(x, a, b, offsets, adapter, base=base, scales=scales)
    assert got.dtype == F32
    tol = (16 + 1.5 * k / 32 + 4.5 * rank / 32) * 2 * U * mag + 20 * U * (want.abs() + mag)
    bad = ~((got.to(D) - want).abs() <= tol)
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[0].tolist(), got[bad][0].item(), want[bad][0].item())
    assert torch.equal(got[of_row < 0], base[of_row < 0])
    assert torch.equal(B.situ_moe_adapters(x, a, b, offsets, adapter, base=base, scales=scales), got)


def test_between_the_products_nothing_overflows():
    """A finite value has finite terms, up to fp32's largest; what is not finite stays so, in its own rows."""
    rows = 300
    x = torch.zeros(rows, 64, dtype=BF, device="cuda")
    x[:, :2] = 1.0
    a = torch.zeros(1, 8, 64, dtype=BF, device="cuda")
    a[:, :, 0], a[:, :, 1] = torch.finfo(BF).max, 1.5 * 2.0 ** 119       # the sum rounds to infinity in bf16
    b = torch.full((1, 8, 8), 2.0 ** -80, dtype=BF, device="cuda")
    x[7, 2], x[9, 3] = float("inf"), float("nan")
    a[:, :, 2] = 1.0
    off, ids = torch.tensor([0, rows], dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    got = B.situ_moe_adapters(x, a, b, off, ids, out_dtype=F32)
    want = 8 * 2.0 ** -80 * (float(a[0, 0, 0]) + 1.5 * 2.0 ** 119)
    keep = torch.ones(rows, dtype=torch.bool, device="cuda")
    keep[[7, 9]] = False
    assert ((got[keep].to(D) - want).abs() <= 64 * U * want).all()
    assert not torch.isfinite(got[7]).any() and torch.isnan(got[9]).all()
