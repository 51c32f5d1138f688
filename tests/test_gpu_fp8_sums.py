"""How the FP8 product with scales per 128 sums large products that cancel.

Every aligned eight of k holds two products of +-P = 2^16 that cancel and six
of 1 to 4, 2^-16 to 2^-14 of P, all of one sign.  The true sum over a block is
96 small products, 216 on average.  An fp32 sum of 128 products keeps it: its
bound (test_gpu_grouped.close) is (8 + 8) 2^-23 of the magnitudes, 32 P and a
little, so 4.  The FP8 matrix instruction drops the small products whole: the
documented bound of bf16 outputs is 7 * 2^-13 of the largest of each eight
more, 16 * 7 * 2^-13 P = 896.
"""

import pytest
import torch

import block_scaled_mxfp4_amd as B
from test_gpu_grouped import BF, D, F8, F32, close, fp8_ref, gen_of, offsets_of

pytestmark = pytest.mark.gpu


def cancelling(g, rows, experts, n, k):
    """E4M3 codes and scales of such sums; k a multiple of 16."""
    small = lambda *s: 1 + torch.randint(0, 8, s, generator=g, device="cuda").float() / 8   # noqa: E731
    a, w = small(rows, k), small(experts, n, k)
    first = torch.randint(0, 8, (k // 8,), generator=g, device="cuda") + 8 * torch.arange(k // 8, device="cuda")
    second = first // 8 * 8 + (first + 3) % 8
    a[:, first], a[:, second] = 256.0, 256.0
    w[:, :, first], w[:, :, second] = 256.0, -256.0
    sa = torch.rand(rows, -(-k // 128), generator=g, device="cuda") + 0.5
    sw = torch.rand(experts, -(-n // 128), -(-k // 128), generator=g, device="cuda") + 0.5
    return a.to(F8).view(torch.uint8), sa, w.to(F8).view(torch.uint8), sw


@pytest.mark.parametrize("counts,n,k", [([4], 300, 640), ([40], 2000, 1152), ([130], 4104, 640), ([700], 1032, 640),
                                        ([2050], 2056, 256), ([4200], 4104, 640), ([60, 0, 45], 520, 1792),
                                        ([3, 5, 0, 2], 72, 272), ([1500, 0, 1, 2700], 4104, 384)])
def test_cancelling_products(counts, n, k):
    g = gen_of(n + k)
    rows = sum(counts)
    a, sa, w, sw = cancelling(g, rows, len(counts), n, k)
    want, mag, eights = fp8_ref(a, sa, w, sw, counts)
    off = offsets_of(counts)
    few = rows <= max(8, 4 * len(counts))
    got = B.situ_moe_matmul_fp8_block128(a, sa, w, sw, offsets=off, out_dtype=F32)
    close(got, want, mag, k, 2.0)
    # what the test is worth: an fp32 sum of such products is far nearer than the bf16 bound
    assert ((got.to(D) - want).abs() < 0.1 * 7 * 2.0 ** -13 * eights).all()
    got = B.situ_moe_matmul_fp8_block128(a, sa, w, sw, offsets=off)
    close(got, want, mag, k, 2.0, None if few else eights)
    if len(counts) == 1:
        for out in (F32, BF):
            got = B.situ_moe_matmul_fp8_block128(a, sa, w[0], sw[0], out_dtype=out)
            close(got, want, mag, k, 2.0, None if few or out == F32 else eights)
