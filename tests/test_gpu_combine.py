"""The combine of a token's expert rows and its gradients against the formulas in
64 bits.

Tolerances.  u = 2^-24.  out: top_k fused multiply-adds in order, within
(top_k + 1) u of the products' magnitudes.  d_weights: a lane's chain of
hidden / 64 multiply-adds and six additions, within (hidden / 64 + 16) u of them.
dy: one product.  bf16 is rounded once more, 2^-8 of the value.
"""

import numpy as np
import pytest
import torch

import block_scaled_mxfp4_amd as B

pytestmark = pytest.mark.gpu

BF, F32, D = torch.bfloat16, torch.float32, torch.float64
U = 2.0 ** -24


def gen_of(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def close(got, want, tol):
    assert got.shape == want.shape
    if got.dtype == BF:
        tol = tol * (1 + 2.0 ** -8) + 2.0 ** -8 * want.abs() + 2.0 ** -133
    bad = ~((got.to(D) - want).abs() <= tol)
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[0].tolist(), got[bad][0].item(), want[bad][0].item())


def table(rng, tokens, k, rows):
    """Rows 0 .. rows - 1 given to as many of the pairs, -1 to the others."""
    inv = np.full(tokens * k, -1, np.int32)
    inv[rng.permutation(tokens * k)[:rows]] = rng.permutation(rows)
    return torch.from_numpy(inv).cuda().view(tokens, k)


def randn(g, rows, cols, dtype, pad=0):
    whole = torch.full((rows, cols + pad), float("nan"), device="cuda")
    whole[:, :cols] = torch.randn(rows, cols, generator=g, device="cuda")
    return whole.to(dtype)[:, :cols]


def gathered(y, inv):
    at = inv.long()
    ok = (at >= 0) & (at < y.shape[0])
    if y.shape[0] == 0:
        return torch.zeros(*inv.shape, y.shape[1], dtype=D, device="cuda"), ok
    return torch.where(ok[..., None], y.to(D)[torch.where(ok, at, 0)], 0.0), ok


def check(y, w, inv, d_out, out_dtype):
    k, hidden = inv.shape[1], y.shape[1]
    rows, ok = gathered(y, inv)
    ww = torch.where(ok, w.to(D), 0.0)
    out = B.situ_moe_combine(y, w, inv, out_dtype=out_dtype)
    assert out.dtype == out_dtype
    close(out, (ww[..., None] * rows).sum(1), (k + 1) * U * (ww[..., None] * rows).abs().sum(1) + 2.0 ** -120)
    kept = torch.full(y.shape, 5.0, dtype=y.dtype, device="cuda")
    dy, dw = B.situ_moe_combine_backward(d_out, y, w, inv, dy=kept)
    d = d_out.to(D)
    close(dw, (d[:, None] * rows).sum(2), (hidden / 64 + 16) * U * (d[:, None] * rows).abs().sum(2) + 2.0 ** -120)
    assert (dw[~ok] == 0).all()
    want = torch.full(y.shape, 5.0, dtype=D, device="cuda")
    t, s = ok.nonzero(as_tuple=True)
    want[inv[t, s].long()] = ww[t, s, None] * d[t]
    close(dy, want, U * want.abs() + 2.0 ** -120)
    return out, dy, dw


@pytest.mark.parametrize("tokens,k,hidden,share,pad", [
    (1, 1, 8, 1.0, 0), (1, 16, 3584, 1.0, 0), (3, 2, 64, 0.5, 8), (17, 16, 3584, 0.125, 16), (65, 8, 1000, 1.0, 0),
    (40, 70, 264, 0.7, 0), (9, 130, 72, 0.3, 8), (500, 6, 520, 0.9, 0), (33, 5, 8200, 0.6, 8), (12, 4, 96, 0.0, 0),
    (9000, 2, 128, 0.5, 0)])
@pytest.mark.parametrize("y_dtype,out_dtype", [(BF, BF), (BF, F32), (F32, BF), (F32, F32)])
def test_combine(tokens, k, hidden, share, pad, y_dtype, out_dtype):
    rng = np.random.RandomState(tokens + hidden)
    g = gen_of(tokens + hidden)
    rows = round(share * tokens * k)
    inv = table(rng, tokens, k, rows)
    y = randn(g, rows, hidden, y_dtype, pad)
    d_out = randn(g, tokens, hidden, out_dtype, pad)
    for wd in (BF, F32):
        w = torch.softmax(torch.randn(tokens, k, generator=g, device="cuda"), 1).to(wd)
        w[inv < 0] = float("nan")                       # weights of pairs elsewhere are nobody's business
        out, dy, dw = check(y, w, inv, d_out, out_dtype)
    if not rows:
        assert not out.any()
    # the flat table, a repeated call
    assert torch.equal(B.situ_moe_combine(y, w, inv.view(-1), out_dtype=out_dtype), out)
    again = B.situ_moe_combine_backward(d_out, y, w, inv.view(-1), dy=dy.clone())
    assert torch.equal(again[0], dy) and torch.equal(again[1], dw)


def test_values_outside_the_rows():
    """Rows of no pair are left alone, whatever they hold; a row may serve two pairs of the sum."""
    g = gen_of(2)
    y = randn(g, 10, 256, BF)
    y[4] = float("nan")
    y[5] = float("inf")
    inv = torch.tensor([[0, 1], [10, 2], [-7, 3], [1 << 30, -1]], dtype=torch.int32, device="cuda")
    w = torch.rand(4, 2, generator=g, device="cuda")
    d = randn(g, 4, 256, BF)
    out, dy, dw = check(y, w, inv, d, F32)
    assert torch.isfinite(out).all() and (out[3] == 0).all() and (dy[4:] == 5).all() and torch.isfinite(dw).all()
    twice = torch.zeros(4, 2, dtype=torch.int32, device="cuda")
    out = B.situ_moe_combine(y, w, twice, out_dtype=F32)
    close(out, w.to(D).sum(1, keepdim=True) * y[0].to(D), 3 * U * w.to(D).sum(1, keepdim=True) * y[0].to(D).abs())


def test_zero_weight_of_a_row_that_is_not_finite():
    """As the formula has it: 0 * inf is NaN, and stays in its token."""
    y = torch.ones(2, 64, dtype=BF, device="cuda")
    y[1] = float("inf")
    inv = torch.tensor([[0], [1]], dtype=torch.int32, device="cuda")
    out = B.situ_moe_combine(y, torch.tensor([[1.0], [0.0]], device="cuda"), inv)
    assert (out[0] == 1).all() and torch.isnan(out[1]).all()


def test_gradients_by_differences():
    g = gen_of(3)
    rng = np.random.RandomState(3)
    tokens, k, hidden = 3, 4, 16
    inv = table(rng, tokens, k, 9)
    y, d = randn(g, 9, hidden, F32), randn(g, tokens, hidden, F32)
    w = torch.rand(tokens, k, generator=g, device="cuda")
    dy, dw = B.situ_moe_combine_backward(d, y, w, inv)

    def value(yy, ww):
        rows, ok = gathered(yy, inv)
        return float(((torch.where(ok, ww, 0.0)[..., None] * rows).sum(1) * d.to(D)).sum())

    h = 1e-4                                            # the sum is linear in each: differences are exact to 1e-11
    for t in range(tokens):
        for s in range(k):
            up, down = w.to(D).clone(), w.to(D).clone()
            up[t, s] += h
            down[t, s] -= h
            assert abs((value(y, up) - value(y, down)) / (2 * h) - dw[t, s].item()) < 1e-5
    for r, c in ((0, 0), (4, 7), (8, 15)):
        up, down = y.to(D).clone(), y.to(D).clone()
        up[r, c] += h
        down[r, c] -= h
        assert abs((value(up, w.to(D)) - value(down, w.to(D))) / (2 * h) - dy[r, c].item()) < 1e-5


def test_in_place():
    g = gen_of(4)
    rng = np.random.RandomState(4)
    inv = table(rng, 50, 8, 300)
    y, d = randn(g, 300, 520, BF), randn(g, 50, 520, BF)
    w = torch.rand(50, 8, generator=g, device="cuda")
    dy, dw = B.situ_moe_combine_backward(d, y, w, inv)
    x = y.clone()
    got = B.situ_moe_combine_backward(d, x, w, inv, dy=x)
    assert got[0] is x and torch.equal(x, dy) and torch.equal(got[1], dw)


def test_past_32_bits():
    rows, hidden = 300_000, 7168                        # y begins its last rows past 2^32 bytes
    y = torch.zeros(rows, hidden, dtype=BF, device="cuda")
    g = gen_of(5)
    at = torch.tensor([[0, 299_999], [299_700, 150_000]], dtype=torch.int32, device="cuda")
    for r in at.flatten().tolist():
        y[r] = torch.randn(hidden, generator=g, device="cuda").to(BF)
    w = torch.rand(2, 2, generator=g, device="cuda")
    small = y[at.flatten().long()].clone()
    here = torch.arange(4, dtype=torch.int32, device="cuda").view(2, 2)
    assert torch.equal(B.situ_moe_combine(y, w, at), B.situ_moe_combine(small, w, here))
    d = randn(g, 2, hidden, BF)
    dy, dw = B.situ_moe_combine_backward(d, y, w, at, dy=y)
    want = B.situ_moe_combine_backward(d, small, w, here)
    assert torch.equal(dw, want[1]) and torch.equal(dy[at.flatten().long()], want[0])


def test_graph_and_streams():
    g = gen_of(6)
    rng = np.random.RandomState(6)
    tokens, k, hidden, rows = 100, 8, 1536, 500
    inv = table(rng, tokens, k, rows)
    y, d = randn(g, rows, hidden, BF), randn(g, tokens, hidden, BF)
    w = torch.rand(tokens, k, generator=g, device="cuda")

    def step(**kw):
        return (B.situ_moe_combine(y, w, inv, **kw), *B.situ_moe_combine_backward(d, y, w, inv, **kw))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for i in range(4):
        inv.copy_(table(rng, tokens, k, rows))
        y.copy_(randn(g, rows, hidden, BF))
        graph.replay()
        torch.cuda.synchronize()
        want = step()
        got = step(stream=side)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(held, want)), i
        assert all(torch.equal(a, b) for a, b in zip(got, want)), i
