"""The activation's gradient for incoming gradients of the type's largest magnitude:
it is what the formula says wherever that is finite, though dh up is not.

Tolerances: those of test_gpu_activation.py, with m up to 100.
"""

import pytest
import torch

import block_scaled_mxfp4_amd as B
from test_gpu_activation import KINDS, U, formulas

pytestmark = pytest.mark.gpu

BF, D = torch.bfloat16, torch.float64
MOST = torch.finfo(BF).max


@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("largest", [-0.75 * MOST, 1e38, -1e30])
def test_large_gradients(kind, largest):
    con = {n: torch.tensor([v], device="cuda") for n, v in zip(KINDS[kind], (4.0, 25.0) if kind == "situ" else (1.7, 0.5))}
    g = torch.tensor([-MOST, -1000, -200, -100, -20, -3, -0.01, 0, 0.5, 3, 20, 40, 100, 1000, MOST], dtype=BF, device="cuda")
    u = torch.tensor([-1e20, -30, -1, -0.001, 0, 0.25, 3, 1000], dtype=BF, device="cuda")
    g, u = (t.reshape(1, -1) for t in torch.meshgrid(g, u, indexing="ij"))                  # 120 columns
    dh = torch.full_like(g, largest)
    d = B.situ_moe_activation_backward(dh, torch.cat([g, u], 1), activation=kind, **con)
    p = [con[n].to(D)[:, None] for n in KINDS[kind]]
    _, wg, wu, mag, _ = formulas(kind, g.to(D), u.to(D), dh.to(D), p)
    floor = 2.0 ** -120 * (1 + u.to(D).abs()) * (1 + dh.to(D).abs()) * (1 + g.to(D).abs().clamp(max=100))
    for got, want, m in ((d[:, :120], wg, mag), (d[:, 120:], wu, wu.abs())):
        over, fits = want.abs() > MOST * (1 + 2.0 ** -10), want.abs() < MOST * (1 - 2.0 ** -10)
        assert torch.isinf(got[over]).all() and torch.equal(got[over] > 0, want[over] > 0)
        tol = (1328 * U * m + floor) * (1 + 2.0 ** -8) + 2.0 ** -8 * want.abs()
        bad = fits & ~((got.to(D) - want).abs() <= tol)
        assert not bad.any(), (g[bad].tolist(), u[bad].tolist(), got[bad].tolist(), want[bad].tolist())


def test_last_normal_sigmoids():
    """Gates down to -87, where sigmoid(g) is fp32's last normal value: h keeps its accuracy with both tanh saturated.
    Tolerance: (6 m + 64) u a factor with m up to 88, and bf16's rounding; nothing on the way is below 2^-126."""
    g = torch.arange(-87, -79, 0.5, device="cuda").to(BF)
    con = dict(situ_beta=torch.tensor([4.0], device="cuda"), situ_linear_beta=torch.tensor([25.0], device="cuda"))
    for up in (1000.0, -300.0, 10.0, MOST):
        both = torch.cat([g, torch.full_like(g, up)])[None].contiguous()
        h = B.situ_moe_activation(both, **con)
        p = [c.to(D)[:, None] for c in con.values()]
        want = formulas("situ", both.to(D)[:, :16], both.to(D)[:, 16:], torch.zeros(1, 16, dtype=D, device="cuda"), p)[0]
        assert ((h.to(D) - want).abs() <= ((12 * 88 + 128) * U + 2.0 ** -8) * want.abs()).all(), (up, h.tolist(), want.tolist())
