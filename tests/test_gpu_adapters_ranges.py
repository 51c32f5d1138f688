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
