"""The gate's sums over a million tokens, and sizes at which a wave adds most.

Tolerances.  u = 2^-24, D the row's span of logits.  A share is within (6 D + 64) u of
its value (test_gpu_router.py derives it).  The grid has at most 768 workgroups of 8
waves, 512 with a bias and over 512 experts: a wave adds at most tokens / 4096 + 1 shares,
then eight waves, up to 768 parts in strides of 64 and their tree add some 40 times
more: a sum of positive terms is off by at most (tokens / 4096 + 100) u of itself beside
its terms.  The loss adds up to 1024 products in trees and rounds some 40 times.
"""

import pytest
import torch

import block_scaled_mxfp4_amd as B

pytestmark = pytest.mark.gpu

F32, BF, D = torch.float32, torch.bfloat16, torch.float64
U = 2.0 ** -24


@pytest.mark.parametrize("experts,top_k,scoring,bias,dtype", [
    (520, 8, "sigmoid", True, F32), (520, 8, "softmax", False, BF), (24, 2, "sigmoid", True, F32), (24, 2, "softmax", False, F32)])
def test_sums_over_a_million_tokens(experts, top_k, scoring, bias, dtype):
    tokens = (1 << 20) + 77
    g = torch.Generator(device="cuda")
    g.manual_seed(experts)
    # all tokens alike but for a little: the additions of a wave all round the same way
    z = (torch.randn(experts, generator=g, device="cuda") + 0.01 * torch.randn(tokens, experts, generator=g, device="cuda")).to(dtype)
    b = 0.1 * torch.randn(experts, generator=g, device="cuda") if bias else None
    ids, weights, counts, prob_sum, loss = B.situ_moe_router(z, top_k, scoring=scoring, bias=b, balance=True)
    assert torch.equal(counts.long(), torch.bincount(ids.flatten().long(), minlength=experts))
    want, span = torch.zeros(experts, dtype=D, device="cuda"), 0.0
    for part in z.split(1 << 17):
        p = part.to(D)
        span = max(span, float((p.amax(1) - p.amin(1)).max()))
        p = torch.softmax(p, 1) if scoring == "softmax" else torch.sigmoid(p)
        want += (p / p.sum(1, keepdim=True)).sum(0)
    tol = (6 * span + 64 + tokens / 4096 + 100) * U
    assert ((prob_sum.to(D) - want).abs() <= tol * want).all()
    c = counts.sum().to(D)
    full = experts * top_k * (counts.to(D) @ want) / (c * c)
    assert abs(float(loss) - float(full)) <= (tol + 80 * U) * float(full)
    again = B.situ_moe_router(z, top_k, scoring=scoring, bias=b, balance=True)
    assert all(torch.equal(x, y) for x, y in zip(again, (ids, weights, counts, prob_sum, loss)))
