"""The steps around the routed products together, as a user runs them: a routed
layer of bf16 experts forward and back (gate, routing tables, grouped products,
activation with its 8-bit copy, combine), and adapters of a batch of requests on
the projection in front of it.

The forward and every gradient are compared with the same layer in 64 bits,
differentiated by autograd, on the choice of experts that the gate made.  The
64-bit layer rounds nothing, so the tolerance is that of the chain's roundings: each
stage rounds its output to bf16 once (2^-8 of the element), and in the way back
gate and up come from 8 bits (2^-4 of the element).  Errors of independent elements
add up as their squares do; a stage's error is taken relative to the norm of the
whole array: 2^-8 a bf16 stage, 2^-4 through the 8-bit copy, and no more than ten
stages lie in a row: 10 * 2^-8 without the copy and with it 10 * 2^-8 + 2 * 2^-4
of the norm.
"""

import numpy as np
import pytest
import torch

import block_scaled_mxfp4_amd as B

pytestmark = pytest.mark.gpu

BF, F32, D = torch.bfloat16, torch.float32, torch.float64


def near(got, want, rel):
    err = (got.to(D) - want).norm().item() / want.norm().item()
    assert err <= rel, err


def tables(ids, experts, top_k):
    """offsets, perm and inv of the layer's own routing."""
    prob = B.make_problem(num_tokens=ids.shape[0], hidden_size=64, intermediate_size=32, num_experts=experts,
                          local_expert_offset=0, local_num_experts=experts, top_k=top_k)
    plan = B.situ_moe_plan(prob)
    ws = B.new_workspace(plan)
    ts = B.SituMoeTensors()
    ts.topk_ids, weights = ids.data_ptr(), torch.zeros(ids.shape, dtype=BF, device="cuda")
    ts.topk_weights = weights.data_ptr()
    B.situ_moe_route(plan, ts, ws)
    view = lambda r, n: B.workspace_view(plan, ws, r, torch.int32, (n,))     # noqa: E731
    return view("offsets", experts + 1).clone(), view("perm", ids.numel()).clone(), view("inv", ids.numel()).clone()


@pytest.mark.parametrize("scoring,activation", [("softmax", "situ"), ("sigmoid", "swiglu")])
@pytest.mark.parametrize("tokens", [1, 37, 600])
def test_training_step(tokens, scoring, activation):
    g = torch.Generator(device="cuda")
    g.manual_seed(tokens)
    E, k, H, I = 24, 4, 256, 128

    def normal(*shape, scale=1.0):
        return (scale * torch.randn(*shape, generator=g, device="cuda")).to(BF)

    x, wr = normal(tokens, H), normal(1, E, H, scale=H ** -0.5)
    w1, w2 = normal(E, 2 * I, H, scale=H ** -0.5), normal(E, H, I, scale=I ** -0.5)
    p0, p1 = 0.5 + torch.rand(E, generator=g, device="cuda"), 0.5 + torch.rand(E, generator=g, device="cuda")
    con = dict(situ_beta=p0, situ_linear_beta=p1) if activation == "situ" else {}
    con["activation"] = activation
    d_out, d_loss = normal(tokens, H), torch.tensor([3.0], device="cuda")
    gate = dict(scoring=scoring, renormalize=True)
    mask = torch.ones(tokens, dtype=torch.bool, device="cuda")
    if tokens > 30:
        mask[-5:] = False                                       # a padded batch

    # forward
    logits = B.situ_moe_grouped_matmul(x, wr, out_dtype=F32)
    ids, weights, counts, prob_sum, loss = B.situ_moe_router(logits, k, mask=mask, balance=True, **gate)
    offsets, perm, inv = tables(ids, E, k)
    pairs = int(offsets[-1])
    perm = perm[:pairs]
    assert torch.equal(counts, offsets.diff())
    gate_up = B.situ_moe_grouped_matmul(x, w1, offsets, pairs=perm, x_div=k)
    h, codes, scales = B.situ_moe_activation(gate_up, offsets=offsets, checkpoint=True, **con)
    y = B.situ_moe_grouped_matmul(h, w2, offsets)
    out = B.situ_moe_combine(y, weights, inv, out_dtype=F32)
    assert not out[~mask].any()

    # the way back: of gate_up and h only the 8-bit copy was kept
    dy, d_weights = B.situ_moe_combine_backward(d_out, y, weights, inv)
    dh = B.situ_moe_grouped_matmul_dgrad(dy, w2, offsets)
    d_gate_up, h_again = B.situ_moe_activation_backward(dh, codes, scales, offsets=offsets, recompute=True, **con)
    dw2 = B.situ_moe_grouped_matmul_wgrad(dy, h_again, offsets)
    dw1 = B.situ_moe_grouped_matmul_wgrad(d_gate_up, x, offsets, pairs=perm, x_div=k)
    dx_rows = torch.zeros(tokens * k, H, dtype=BF, device="cuda")
    B.situ_moe_grouped_matmul_dgrad(d_gate_up, w1, offsets, pairs=perm, out_div=1, out=dx_rows)
    d_logits = B.situ_moe_router_backward(logits, ids, d_weights, mask=mask, counts=counts, d_loss=d_loss, out_dtype=BF, **gate)
    dwr = B.situ_moe_grouped_matmul_wgrad(d_logits, x)
    dx = dx_rows.view(tokens, k, H).float().sum(1) + B.situ_moe_grouped_matmul_dgrad(d_logits, wr).float()

    # the same layer in 64 bits
    xd, wrd, w1d, w2d = (t.to(D).requires_grad_() for t in (x, wr[0], w1, w2))
    z = xd @ wrd.t()
    p = torch.softmax(z, 1) if scoring == "softmax" else torch.sigmoid(z)
    e = ids.long().clamp(min=0)
    wd = p.gather(1, e)
    wd = wd / wd.sum(1, keepdim=True) * mask[:, None]
    share = p / p.sum(1, keepdim=True) * mask[:, None]
    c = counts.to(D)
    loss64 = E * k * (c @ share.sum(0)) / c.sum() ** 2
    o = 0
    for s in range(k):
        gu = torch.einsum("th,tgh->tg", xd, w1d[e[:, s]])
        a, u = gu[:, :I], gu[:, I:]
        if activation == "situ":
            b, lb = p0.to(D)[e[:, s], None], p1.to(D)[e[:, s], None]
            hh = b * torch.tanh(a / b) * torch.sigmoid(a) * lb * torch.tanh(u / lb)
        else:
            hh = a * torch.sigmoid(a) * u
        o = o + wd[:, s, None] * torch.einsum("ti,thi->th", hh, w2d[e[:, s]])
    ((o * d_out.to(D) * mask[:, None]).sum() + 3.0 * loss64).backward()
    assert abs(loss.item() - loss64.item()) <= 1e-4 * loss64.item()      # z is fp32: 2^-24 H^0.5 of its terms
    near(out, o.detach() * mask[:, None], 10 * 2.0 ** -8)
    for got, want in ((dw2, w2d.grad), (dw1, w1d.grad), (dwr[0], wrd.grad), (dx, xd.grad)):
        near(got, want, 10 * 2.0 ** -8 + 2 * 2.0 ** -4)


def test_adapters_in_front_of_the_gate():
    """A batch of requests through an adapted projection, then the gate: every request as if it were alone."""
    g = torch.Generator(device="cuda")
    g.manual_seed(2)
    counts, H, E = [1, 1, 40, 0, 7, 1], 512, 64
    rows = sum(counts)
    off = torch.tensor([0] + list(np.cumsum(counts)), dtype=torch.int32, device="cuda")
    adapter = torch.tensor([0, -1, 1, 0, 2, 1], dtype=torch.int32, device="cuda")
    x = torch.randn(rows, H, generator=g, device="cuda").to(BF)
    w = (torch.randn(1, H, H, generator=g, device="cuda") / H ** 0.5).to(BF)
    a = (torch.randn(3, 16, H, generator=g, device="cuda") / H ** 0.5).to(BF)
    b = (torch.randn(3, H, 16, generator=g, device="cuda") / 4).to(BF)
    wr = torch.randn(1, E, H, generator=g, device="cuda").to(BF)
    y = B.situ_moe_grouped_matmul(x, w)
    B.situ_moe_adapters(x, a, b, off, adapter, base=y, out=y)
    ids, _ = B.situ_moe_router(B.situ_moe_grouped_matmul(y, wr, out_dtype=F32), 4)
    plain = B.situ_moe_grouped_matmul(x, w)
    for q, (lo, hi) in enumerate(zip(off.tolist()[:-1], off.tolist()[1:])):
        i = int(adapter[q])
        want = plain[lo:hi].to(D)
        mag = want.abs()
        if i >= 0:
            want = want + (x[lo:hi].to(D) @ a[i].to(D).t()) @ b[i].to(D).t()
            mag = mag + (x[lo:hi].to(D).abs() @ a[i].to(D).abs().t()) @ b[i].to(D).abs().t()
        assert ((y[lo:hi].to(D) - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -15 * mag).all(), q
    z = y.to(D) @ wr[0].to(D).t()
    mag = y.to(D).abs() @ wr[0].to(D).abs().t()
    assert (z.gather(1, ids[:, :1].long())[:, 0] >= z.amax(1) - 2.0 ** -18 * mag.amax(1)).all()     # fp32 sums of 512
