"""Adapters at the ends of their ranges: values near the types' largest.

Tolerances.  u = 2^-24: bf16 rounds the result once, 2^-8 of it, beside the 64 u of
a few fp32 sums and the 2^-16 that two terms may lose.
"""

import pytest
import torch

import block_scaled_mxfp4_amd as B

pytestmark = pytest.mark.gpu

BF, D = torch.bfloat16, torch.float64
U = 2.0 ** -24


@pytest.mark.parametrize("rank", [8, 16, 40])
@pytest.mark.parametrize("rows", [3, 300])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_first_product_past_the_types_largest(rows, rank, sign):
    """a x between bf16's largest value and fp32's is finite, and so is what b makes of it, in few rows and in many."""
    x = torch.zeros(rows, 64, dtype=BF, device="cuda")
    x[:, :2] = sign
    a = torch.zeros(1, rank, 64, dtype=BF, device="cuda")
    a[:, :, 0], a[:, :, 1] = torch.finfo(BF).max, 1.5 * 2.0 ** 119       # the sum rounds to infinity in bf16
    b = torch.full((1, 24, rank), 2.0 ** -80, dtype=BF, device="cuda")
    off, ids = torch.tensor([0, rows], dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    got = B.situ_moe_adapters(x, a, b, off, ids)
    want = sign * rank * 2.0 ** -80 * (float(a[0, 0, 0]) + 1.5 * 2.0 ** 119)
    assert got.dtype == BF and ((got.to(D) - want).abs() <= (2.0 ** -8 + 64 * U + 2.0 ** -16) * abs(want)).all()


def test_rows_past_32_bits():
    """Rows of x, then of base and out, that begin past 2^32 bytes, each within the bound of its own magnitudes: with M
    what the two products add, (32 + 1.5 k / 32 + 4.5 rank / 32) 2 u M, for a bf16 out 2^-16 of M for the two terms, 20
    roundings of what is added, and the last one."""
    rows, rank = 310_000, 16
    g = torch.Generator(device="cuda")
    g.manual_seed(6)

    def run(k, n, dtype):
        x = torch.zeros(rows, k, dtype=BF, device="cuda")
        x[-40:] = torch.randn(40, k, generator=g, device="cuda").to(BF)
        a = (k ** -0.5 * torch.randn(2, rank, k, generator=g, device="cuda")).to(BF)
        b = (rank ** -0.5 * torch.randn(2, n, rank, generator=g, device="cuda")).to(BF)
        base = torch.zeros(rows, n, dtype=dtype, device="cuda")
        base[-40:] = torch.randn(40, n, generator=g, device="cuda").to(dtype)
        last, ids = x[-40:].to(D), torch.tensor([0] * 10 + [1] * 30, device="cuda")
        want, mag = base[-40:].to(D), torch.zeros(40, n, dtype=D, device="cuda")
        for i in range(2):
            on = ids == i
            want[on] += (last[on] @ a[i].to(D).t()) @ b[i].to(D).t()
            mag[on] = (last[on].abs() @ a[i].to(D).abs().t()) @ b[i].to(D).abs().t()
        out = B.situ_moe_adapters(x, a, b, torch.tensor([0, rows - 30, rows], dtype=torch.int32, device="cuda"),
                                  torch.tensor([0, 1], dtype=torch.int32, device="cuda"), base=base, out=base)
        tol = (32 + 1.5 * k / 32 + 4.5 * rank / 32) * 2 * U * mag + 20 * U * (want.abs() + mag)
        if dtype == BF:
            tol = (tol + 2.0 ** -16 * mag) * (1 + 2.0 ** -8) + 2.0 ** -8 * want.abs()
        assert not out[:-40].any()
        assert ((out[-40:].to(D) - want).abs() <= tol).all()

    run(7168, 64, torch.float32)
    run(64, 7168, BF)
    run(64, 3584, torch.float32)
