"""SiTU with betas from far below 1 to infinity: the activation, what the gradient
recomputes of it and the gradient against the formulas in 64 bits.

Tolerances: those of test_gpu_activation.py.  They hold for every beta, since
|b tanh(x / b)| is at most |x|: a value below fp32's smallest normal one costs at most
2^-126 times the product of the other factors, which is below (1 + |g|) (1 + |u|) (1 +
|dh|), a few times; and what an underflow of x / b changes in tanh is squared.
"""

import numpy as np
import pytest
import torch

import block_scaled_mxfp4_amd as B
from test_gpu_activation import close, formulas, gen_of, widened

pytestmark = pytest.mark.gpu

BF, D = torch.bfloat16, torch.float64
INF = float("inf")
PAIRS = [(4.0, 25.0), (0.02, 50.0), (1e3, 1e-3), (1e-3, 1e3), (-4.0, 25.0), (4.0, -25.0), (1e18, 1e18), (1e20, 1e20),
         (1e30, 1e30), (3e38, 3e38), (1.0, 3e38), (3e38, 1.0), (INF, INF), (-INF, 2.0), (1.0, INF)]


def both(g, u, dh, b, l):
    """formulas(), where an infinite beta is one that 64 bits cannot tell from it."""
    return formulas("situ", g, u, dh, [torch.where(t.isinf(), 1e150, t) for t in (b, l)])


@pytest.mark.parametrize("spread", [0.01, 1.0, 30.0])
@pytest.mark.parametrize("inner", [8, 136, 384])
def test_betas(inner, spread):
    g = gen_of(inner)
    rng = np.random.RandomState(inner)
    counts = rng.randint(1, 40, len(PAIRS))
    rows = int(counts.sum())
    off = torch.tensor([0] + list(np.cumsum(counts)), dtype=torch.int32, device="cuda")
    con = {n: torch.tensor([p[i] for p in PAIRS], device="cuda") for i, n in enumerate(("situ_beta", "situ_linear_beta"))}
    of_row = torch.repeat_interleave(torch.arange(len(PAIRS), device="cuda"), off.diff().long())
    b, l = (c.to(D)[of_row, None] for c in con.values())
    wide = spread * torch.exp(torch.randn(rows, 1, generator=g, device="cuda"))
    gate_up = (torch.randn(rows, 2 * inner, generator=g, device="cuda") * wide).to(BF)
    dh = torch.randn(rows, inner, generator=g, device="cuda").to(BF)
    kw = dict(offsets=off, **con)

    def against(gu, h, again, d):
        gate, up = gu[:, :inner], gu[:, inner:]
        want, dg, du, mag, m = both(gate, up, dh.to(D), b, l)
        factors = (1 + gate.abs()) * (1 + up.abs())
        for got in (h, again):
            if got is not None:
                close(got, want, want.abs(), m, factors)
        factors = factors * (1 + dh.to(D).abs())
        close(d[:, :inner], dg, mag, m, factors)
        close(d[:, inner:], du, du.abs(), m, factors)

    h, codes, scales = B.situ_moe_activation(gate_up, checkpoint=True, **kw)
    assert torch.equal(B.situ_moe_activation(gate_up, **kw), h)
    d, again = B.situ_moe_activation_backward(dh, gate_up, recompute=True, **kw)
    against(gate_up.to(D), h, again, d)
    d, again = B.situ_moe_activation_backward(dh, codes, scales, recompute=True, **kw)
    against(widened(codes, scales, inner), None, again, d)


def test_without_saturation_it_is_swiglu():
    """Infinite betas: g sigmoid(g) u."""
    g = gen_of(5)
    gate_up = torch.randn(50, 512, generator=g, device="cuda").to(BF)
    dh = torch.randn(50, 256, generator=g, device="cuda").to(BF)
    inf = torch.full((1,), INF, device="cuda")
    con = dict(situ_beta=inf, situ_linear_beta=inf)
    want = B.situ_moe_activation_backward(dh, gate_up, activation="swiglu", recompute=True)
    got = B.situ_moe_activation_backward(dh, gate_up, recompute=True, **con)
    h = B.situ_moe_activation(gate_up, **con)
    # each is within 200 u of the formula, dg within that of magnitudes of at most 2.5 |dh u|, and rounded by 2^-8
    mag = torch.cat([2.5 * (dh * gate_up[:, 256:]).abs(), want[0][:, 256:].abs()], 1).double()
    for a, w, m in ((got[0], want[0], mag), (got[1], want[1], want[1].abs().double()), (h, want[1], want[1].abs().double())):
        assert ((a.double() - w.double()).abs() <= 2 * 2.0 ** -8 * w.double().abs() + 400 * 2.0 ** -24 * m + 2.0 ** -120).all()


@pytest.mark.parametrize("betas", [(1.7, 25.0), (1e20, 1e20), (1e35, 2.0), (2.0, 1e35), (1e35, 1e35), (2.0 ** 123, 2.0 ** 123),
                                   (3e38, 3e38), (INF, INF)])
def test_lowest_values(betas):
    """Gates and ups of the type's largest magnitudes and infinite ones: the limits, with any betas."""
    low = torch.finfo(BF).min
    con = dict(zip(("situ_beta", "situ_linear_beta"), (torch.tensor([v], device="cuda") for v in betas)))
    vals = torch.tensor([low, -1e20, -1000.0, 1.0, 3.0, 2.0 ** 21, 1e20, 1e33, -low], dtype=BF, device="cuda")
    g, u = torch.meshgrid(vals, torch.cat([vals, torch.tensor([0.0, 1e-3, -1e-10], dtype=BF, device="cuda")]), indexing="ij")
    g, u = (t[:, None].expand(-1, 2, -1).reshape(1, -1) for t in (g, u))                  # 216 columns
    dh = torch.full_like(g, -0.5)
    both_ = torch.cat([g, u], 1)
    h = B.situ_moe_activation(both_, **con)
    d, again = B.situ_moe_activation_backward(dh, both_, recompute=True, **con)
    # past 2^123 a beta is taken for 2^123
    p = [torch.tensor([[min(float(torch.tensor(abs(v))), 2.0 ** 123)]], dtype=D, device="cuda") for v in betas]
    wh, wg, wu, mag, _ = formulas("situ", g.to(D), u.to(D), dh.to(D), p)
    n = g.shape[1]
    for got, want, m in ((h, wh, wh.abs()), (again, wh, wh.abs()), (d[:, :n], wg, mag), (d[:, n:], wu, wu.abs())):
        over = want.abs() > torch.finfo(BF).max * (1 + 2.0 ** -10)
        assert torch.equal(got[over].float().sign(), want[over].float().sign()) and torch.isinf(got[over]).all()
        fits = want.abs() < torch.finfo(BF).max * (1 - 2.0 ** -10)
        # arguments of exponentials up to 100 (past it they are 0): (12 * 100 + 128) u; 2^-126 of up, and of the gate's 100
        tol = 1328 * 2.0 ** -24 * m + 2.0 ** -8 * want.abs() + 2.0 ** -120 * 100 * (1 + u.to(D).abs())
        bad = fits & ~((got.to(D) - want).abs() <= tol)
        assert not bad.any(), (betas, g[bad].tolist(), u[bad].tolist(), got[bad].tolist(), want[bad].tolist())
