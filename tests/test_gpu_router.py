"""The gate, its balance loss and its gradient against the formulas in 64 bits.

Tolerances.  u = 2^-24.  A score is e^d with |d| up to D (the row's span of
logits): the difference, its product with log2 e and that constant each round
once, D of 3 u in the exponent; the exponential, reciprocal and product add 8 u.
A share divides by a sum of up to 1024 positive scores in a tree of at most 24
additions: (6 D + 64) u relative covers it, and scores below fp32's smallest
normal number may be lost: 2^-120 of the largest share, 1.  A sum over tokens adds at
most tokens / 8192 + 100 additions of positive terms.  A gradient is off by as much
relative to the magnitudes it adds.  A bf16 output is rounded once more: 2^-8 of
the value.
"""

import numpy as np
import pytest
import torch

import block_scaled_mxfp4_amd as B

pytestmark = pytest.mark.gpu

BF, F32, D = torch.bfloat16, torch.float32, torch.float64
U = 2.0 ** -24
NEG = float("-inf")


def gen_of(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def logits_of(g, tokens, experts, dtype, pad=0, scale=1.0):
    whole = torch.full((tokens, experts + pad), float("nan"), device="cuda")
    whole[:, :experts] = scale * torch.randn(tokens, experts, generator=g, device="cuda")
    return whole.to(dtype)[:, :experts]


def choose(z, k, bias=None, mask=None):
    """Ids by repeated search in 64 bits: the largest left, the lowest of equals; -1 where none is left."""
    z = z.to(D)
    key = z.clone() if bias is None else torch.sigmoid(z) + bias.to(D)
    out = torch.isnan(z) | (z == NEG)
    if bias is not None:
        out = out | torch.isnan(key) | (key == NEG)
    if mask is not None:
        out = out | ~mask.bool()[:, None]
    key[out] = NEG
    left = ~out
    ids = torch.full((z.shape[0], k), -1, dtype=torch.long, device="cuda")
    for j in range(k):
        best = torch.where(left, key, NEG).amax(1, keepdim=True)
        hit = left & (key == best)
        some = hit.any(1)
        at = hit.to(torch.int8).argmax(1)
        ids[some, j] = at[some]
        left[some, at[some]] = False
    return ids


def forward(z, ids, scoring, renormalize, scale, mask=None):
    """weights, P in 64 bits."""
    z = z.to(D)
    live = (~(torch.isnan(z) | (z == NEG))).any(1)
    if mask is not None:
        live = live & mask.bool()
    z = torch.where(live[:, None], z, 0.0)
    logs = torch.nn.functional.logsigmoid(z) if scoring == "sigmoid" else z - z.amax(1, keepdim=True)
    p = torch.exp(logs - logs.amax(1, keepdim=True))            # the largest first: log values of 1e38 hold no sum
    total = p.sum(1, keepdim=True)
    p = p / total
    if scoring == "softmax":
        logs = logs - torch.log(total)
    chosen = torch.where(ids >= 0, logs.gather(1, ids.clamp(min=0)), NEG)
    if renormalize:
        top = chosen.amax(1, keepdim=True)
        e = torch.exp(chosen - torch.where(top > NEG, top, 0.0))
        w = e / e.sum(1, keepdim=True).clamp(min=1e-300)
    else:
        w = torch.exp(chosen)
    return scale * w * live[:, None], p * live[:, None], live


def span(z):
    z = z.to(D)
    z = torch.where(torch.isfinite(z), z, 0.0)
    return min(float((z.amax(1) - z.amin(1)).max()) if z.numel() else 0.0, 100.0) + float(z.abs().max().clamp(max=100.0))


def check(got, want, rel, floor):
    assert got.shape == want.shape
    tol = rel * want.abs() + floor
    if got.dtype == BF:
        tol = tol * (1 + 2.0 ** -8) + 2.0 ** -8 * want.abs() + 2.0 ** -133
    bad = ~((got.to(D) - want).abs() <= tol)
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[0].tolist(), got[bad][0].item(), want[bad][0].item())


def run(z, k, scoring="softmax", bias=None, renormalize=True, scale=1.0, mask=None, **kw):
    out = B.situ_moe_router(z, k, scoring=scoring, bias=bias, renormalize=renormalize, scale=scale, mask=mask,
                            balance=True, packed=True, **kw)
    ids, weights, packed, counts, prob_sum, loss = out
    T, E = z.shape
    want = choose(z, k, bias, mask)
    assert torch.equal(ids.long(), want), (ids.long() != want).nonzero()[:3].tolist()
    w, p, live = forward(z, want, scoring, renormalize, scale, mask)
    rel = (6 * span(z) + 64) * U
    check(weights, w, rel, abs(scale) * 2.0 ** -120)
    hits = torch.zeros(E + 1, dtype=torch.long, device="cuda")
    hits.index_add_(0, torch.where(want < 0, E, want).flatten(), torch.ones(T * k, dtype=torch.long, device="cuda"))
    assert torch.equal(counts.long(), hits[:E])
    rel = rel + (T / 8192 + 100) * U
    check(prob_sum, p.sum(0), rel, T * 2.0 ** -120)
    c = hits[:E].sum().to(D)
    want_loss = E * k * (hits[:E].to(D) @ p.sum(0)) / (c * c) if c > 0 else torch.zeros((), dtype=D, device="cuda")
    check(loss, want_loss.view(1), rel + 100 * U, 2.0 ** -100)
    # the packed form holds the bf16 weight and the id
    wb = weights.to(BF).view(torch.int16).long() & 0xffff
    assert torch.equal(packed.long() & 0xffffffff, wb << 16 | (ids.long() & 0xffff))
    # without the loss: the same choice and weights, bit for bit
    plain = B.situ_moe_router(z, k, scoring=scoring, bias=bias, renormalize=renormalize, scale=scale, mask=mask, **kw)
    assert len(plain) == 2 and torch.equal(plain[0], ids) and torch.equal(plain[1], weights)
    return out


MODES = [("softmax", False), ("sigmoid", False), ("sigmoid", True)]


@pytest.mark.parametrize("scoring,biased", MODES)
@pytest.mark.parametrize("tokens,experts,k,pad", [
    (1, 1, 1, 0), (1, 896, 16, 0), (3, 7, 2, 0), (33, 64, 8, 3), (40, 65, 24, 0), (300, 100, 6, 4), (129, 128, 64, 0),
    (70, 160, 1, 1), (65, 256, 8, 0), (50, 384, 33, 8), (31, 513, 16, 0), (257, 896, 16, 4), (20, 1023, 64, 1),
    (17, 1024, 8, 0), (9000, 32, 4, 0)])
def test_router(tokens, experts, k, pad, scoring, biased):
    g = gen_of(tokens + experts)
    for dtype in (F32, BF):
        z = logits_of(g, tokens, experts, dtype, pad, 2.0)
        bias = 0.2 * torch.randn(experts, generator=g, device="cuda") if biased else None
        run(z, k, scoring, bias, True, 2.5)
        run(z, k, scoring, bias, False, 1.0, weights_dtype=F32)


@pytest.mark.parametrize("scoring,biased", MODES)
def test_router_masks(scoring, biased):
    """Padded tokens that hold NaN, experts closed by -inf (more than top_k leaves open), the type's lowest value,
    rows with nothing to choose, batches without a token."""
    g = gen_of(5)
    T, E, k = 203, 112, 8
    bias = 0.2 * torch.randn(E, generator=g, device="cuda") if biased else None
    for dtype in (F32, BF):
        z = logits_of(g, T, E, dtype)
        mask = torch.rand(T, generator=g, device="cuda") < 0.7
        mask[:8] = True
        z[~mask] = float("nan")
        z[0] = NEG                              # nothing to choose
        z[1, 5:] = NEG                          # five experts for eight places
        z[2] = torch.finfo(dtype).min           # all the lowest value: equals
        z[3, ::2] = torch.finfo(dtype).min
        z[4, ::2] = NEG
        for m in (mask, mask.to(torch.uint8)):
            ids, w, *_ = run(z, k, scoring, bias, True, 1.0, m)
        assert (ids[0] == -1).all() and (w[0] == 0).all() and (ids[1, 5:] == -1).all()
        _, _, _, counts, prob_sum, loss = run(z, k, scoring, bias, True, 1.0, torch.zeros_like(mask))
        assert loss.item() == 0 and not counts.any() and not prob_sum.any()
        empty = B.situ_moe_router(z[:0], k, scoring=scoring, bias=bias, balance=True)
        assert empty[0].shape == (0, k) and empty[4].item() == 0 and not empty[2].any() and not empty[3].any()


def test_router_equals():
    """Rows of equals, and of bf16 values with many, choose the lowest ids."""
    for E, k in ((8, 3), (64, 64), (200, 5), (896, 16), (1024, 64)):
        z = torch.zeros(40, E, device="cuda")
        z[::3] = -0.0
        z[1, E // 2:] = -0.0
        run(z, k)
        run(z, k, "sigmoid", torch.zeros(E, device="cuda"))
        z = torch.randn(40, E, generator=gen_of(E), device="cuda").round().to(BF)
        run(z, k)
        run(z, k, "sigmoid")
        run(z, k, "sigmoid", (0.1 * torch.randn(E, generator=gen_of(E), device="cuda")).round(decimals=1))


def test_router_near_scores():
    """Scores with a bias that differ by less than fp32 holds: only 64 bits tell their order."""
    g = gen_of(9)
    E, k = 896, 16
    z = torch.randn(200, E, generator=g, device="cuda")
    bias = (0.9 - torch.sigmoid(z[0].to(D))).float()            # row 0: all sums next to 0.9
    run(z, k, "sigmoid", bias)
    z[:] = 20 + torch.rand(200, E, generator=g, device="cuda")  # sigmoids next to 1, all within 3e-9
    run(z, k, "sigmoid", torch.zeros(E, device="cuda"))
    run(z, k, "sigmoid", 1000 * torch.ones(E, device="cuda"))


def test_router_far_scores():
    """Scores that underflow: renormalized weights and shares stay right."""
    g = gen_of(10)
    E, k = 300, 8
    z = -200 + 3 * torch.randn(64, E, generator=g, device="cuda")
    run(z, k, "sigmoid")
    run(z, k, "softmax")
    bias = torch.zeros(E, device="cuda")
    bias[:k] = 5.0                                              # chosen by their bias, though their scores are the least
    z[:, :k] -= 150
    run(z, k, "sigmoid", bias)
    z = 80 * torch.randn(64, E, generator=g, device="cuda")
    run(z, k, "softmax")
    bias[3], bias[4], bias[5] = NEG, float("inf"), float("nan")
    ids, *_ = run(torch.randn(64, E, generator=g, device="cuda"), k, "sigmoid", bias)
    assert not ((ids == 3) | (ids == 5)).any() and (ids[:, 0] == 4).all()


@pytest.mark.parametrize("size", [2.0 ** 19, 2.0 ** 20, 2.0 ** 21, 1e8, 2e9, 1e10, 1e20, 2.0 ** 100, 1e38])
def test_router_large_logits(size):
    """Logits far from 0 (equals, or neighbours that differ by one step of fp32) have the scores of their differences."""
    g = gen_of(12)
    T, E, k = 40, 200, 8
    step = size * 2.0 ** -23
    for sign in (1, -1):
        z = sign * (size - step * torch.randint(0, 4, (T, E), generator=g, device="cuda").to(D))
        z[0] = sign * size
        z[1, 5:] = -size
        z = z.float()
        for scoring in ("softmax", "sigmoid"):
            for renormalize in (True, False):
                ids, _, _, counts, _, _ = run(z, k, scoring, None, renormalize, 1.0, weights_dtype=F32)
                dw = torch.randn(T, k, generator=g, device="cuda")
                check_backward(z, ids, dw, scoring, renormalize, 1.0, None, counts, torch.ones(1, device="cuda"))


def test_router_nan():
    """A NaN is never chosen, and shows in the loss; other rows' ids and weights are their own."""
    z = torch.randn(70, 96, generator=gen_of(11), device="cuda")
    want = B.situ_moe_router(z, 4, balance=True)
    z[7, 3] = float("nan")
    got = B.situ_moe_router(z, 4, balance=True)
    assert not (got[0][7] == 3).any() and torch.isnan(got[4]).all()
    keep = torch.arange(70, device="cuda") != 7
    assert torch.equal(got[0][keep], want[0][keep]) and torch.equal(got[1][keep], want[1][keep])


# ------------------------------------------------------------------ gradient

def backward64(z, ids, dw, scoring, renormalize, scale, mask, counts, d_loss):
    """The gradient, and the magnitudes it adds."""
    T, E = z.shape
    k = ids.shape[1]
    w, p, live = forward(z, ids, scoring, renormalize, 1.0, mask)
    held = (ids >= 0) & live[:, None]
    at = ids.clamp(min=0)
    dw = torch.where(held, scale * dw.to(D), 0.0)
    g = torch.zeros(E, dtype=D, device="cuda")
    if counts is not None and counts.sum() > 0:
        c = counts.to(D)
        g = float(d_loss) * E * k * c / c.sum() ** 2
    pg = (p * g).sum(1, keepdim=True)
    dz = p * (g - pg)
    mag = p * (g.abs() + (p * g.abs()).sum(1, keepdim=True))
    w = torch.where(held, w, 0.0)
    if renormalize:
        x = w * (dw - (w * dw).sum(1, keepdim=True))
        xm = w * (dw.abs() + (w * dw.abs()).sum(1, keepdim=True))
    else:
        x, xm = w * dw, (w * dw).abs()
        if scoring == "softmax":
            dz = dz - p * x.sum(1, keepdim=True)
            mag = mag + p * xm.sum(1, keepdim=True)
    dz = dz.scatter_add(1, at, torch.where(held, x, 0.0))
    mag = mag.scatter_add(1, at, torch.where(held, xm, 0.0))
    if scoring == "sigmoid":
        left = torch.sigmoid(-torch.where(live[:, None], z.to(D), 0.0))
        dz, mag = dz * left, mag * left
    return dz * live[:, None], mag * live[:, None]


def check_backward(z, ids, dw, scoring, renormalize, scale, mask, counts, d_loss, **kw):
    got = B.situ_moe_router_backward(z, ids, dw, scoring=scoring, renormalize=renormalize, scale=scale, mask=mask,
                                     counts=counts, d_loss=d_loss, **kw)
    zero = torch.zeros(ids.shape, device="cuda")
    want, mag = backward64(z, ids.long(), zero if dw is None else dw, scoring, renormalize, scale, mask, counts,
                           0.0 if d_loss is None else d_loss)
    tol = (8 * span(z) + 128) * U * mag + 2.0 ** -110 * (1 + mag.max())
    if got.dtype == BF:
        tol = tol * (1 + 2.0 ** -8) + 2.0 ** -8 * want.abs() + 2.0 ** -133
    bad = ~((got.to(D) - want).abs() <= tol)
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[0].tolist(), got[bad][0].item(), want[bad][0].item())
    return got


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [True, False])
@pytest.mark.parametrize("tokens,experts,k,pad", [(1, 1, 1, 0), (1, 896, 16, 0), (5, 7, 2, 0), (33, 64, 8, 3),
                                                  (300, 100, 6, 4), (129, 128, 64, 0), (65, 256, 8, 0), (50, 384, 33, 8),
                                                  (31, 513, 16, 0), (257, 896, 16, 4), (20, 1023, 64, 1), (9001, 32, 4, 0)])
def test_backward(tokens, experts, k, pad, renormalize, scoring):
    g = gen_of(tokens * 7 + experts)
    for dtype in (F32, BF):
        z = logits_of(g, tokens, experts, dtype, pad, 2.0)
        ids, _, counts, _, _ = B.situ_moe_router(z, k, scoring=scoring, balance=True)
        dw = torch.randn(tokens, k, generator=g, device="cuda")
        dl = torch.tensor([0.3 * tokens], device="cuda")
        check_backward(z, ids, dw, scoring, renormalize, 2.5, None, counts, dl)
        check_backward(z, ids, dw, scoring, renormalize, 1.0, None, None, None, out_dtype=F32)
        check_backward(z, ids, None, scoring, renormalize, 1.0, None, counts, dl, out_dtype=BF)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [True, False])
def test_backward_masks(scoring, renormalize):
    g = gen_of(21)
    T, E, k = 150, 112, 8
    for dtype in (F32, BF):
        z = logits_of(g, T, E, dtype)
        mask = torch.rand(T, generator=g, device="cuda") < 0.7
        mask[:8] = True
        z[~mask] = float("nan")
        z[0] = NEG
        z[1, 5:] = NEG
        z[2] = torch.finfo(dtype).min
        z[3, ::2] = torch.finfo(dtype).min
        z[5, :] = -150
        ids, _, counts, _, _ = B.situ_moe_router(z, k, scoring=scoring, mask=mask, balance=True)
        dw = torch.randn(T, k, generator=g, device="cuda")
        dw[ids < 0] = float("nan")                              # nobody's
        dl = torch.tensor([2.0], device="cuda")
        got = check_backward(z, ids, dw, scoring, renormalize, 1.0, mask, counts, dl)
        assert (got[~mask] == 0).all() and (got[0] == 0).all()
        # ids that are not the largest, one of them twice, and ids outside the experts
        other = torch.randint(0, E, (T, k), generator=g, device="cuda", dtype=torch.int32)
        other[:, 1] = other[:, 0]
        other[6, 2], other[7, 3] = E, -5
        want = torch.where((other >= 0) & (other < E), other, -1)
        dw = torch.randn(T, k, generator=g, device="cuda")
        zf = torch.where(torch.isfinite(z), z, 0.0).to(dtype)
        a = B.situ_moe_router_backward(zf, other, dw, scoring=scoring, renormalize=renormalize, mask=mask)
        b = check_backward(zf, want, dw, scoring, renormalize, 1.0, mask, None, None)
        assert torch.equal(a, b)
        # no token routed: the loss has no gradient
        zero = torch.zeros_like(counts)
        assert not B.situ_moe_router_backward(zf, ids, counts=zero, d_loss=dl, scoring=scoring).any()


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [True, False])
def test_backward_by_differences(scoring, renormalize):
    """Against central differences of the forward formulas in 64 bits."""
    g = gen_of(31)
    T, E, k = 3, 12, 4
    z = logits_of(g, T, E, F32)
    ids, _, counts, _, _ = B.situ_moe_router(z, k, scoring=scoring, balance=True)
    dw = torch.randn(T, k, generator=g, device="cuda")
    dl = torch.tensor([1.7], device="cuda")
    got = B.situ_moe_router_backward(z, ids, dw, scoring=scoring, renormalize=renormalize, scale=1.5, counts=counts, d_loss=dl)

    def value(zz):
        w, p, _ = forward(zz, ids.long(), scoring, renormalize, 1.5)
        c = counts.to(D)
        return float((w * dw.to(D)).sum() + dl.to(D)[0] * E * k * (c @ p.sum(0)) / c.sum() ** 2)

    h = 1e-5
    for t in range(T):
        for e in range(E):
            up, down = z.to(D).clone(), z.to(D).clone()
            up[t, e] += h
            down[t, e] -= h
            d = (value(up) - value(down)) / (2 * h)
            assert abs(d - got[t, e].item()) < 1e-5, (t, e, d, got[t, e].item())     # 64-bit differences: 1e-10


# --------------------------------------------------------------------- calls

def test_router_repeats_and_outputs():
    """Given outputs are filled, a repeated call gives the same bits, strided logits are read in place."""
    g = gen_of(40)
    T, E, k = 4099, 896, 16
    z = logits_of(g, T, E, F32, 5)
    i32 = dict(dtype=torch.int32, device="cuda")
    outs = dict(ids=torch.empty(T, k, **i32), weights=torch.empty(T, k, device="cuda"), packed=torch.empty(T, k, **i32),
                counts=torch.empty(E, **i32), prob_sum=torch.empty(E, device="cuda"), loss=torch.empty(1, device="cuda"))
    ws = torch.empty(64 << 20, dtype=torch.uint8, device="cuda").fill_(255)
    first = [t.clone() for t in B.situ_moe_router(z, k, workspace=ws, **outs)]
    for i in range(5):
        got = B.situ_moe_router(z, k, workspace=ws, **outs)
        assert all(a is b for a, b in zip(got, outs.values()))
        assert all(torch.equal(a, b) for a, b in zip(got, first)), i
    fresh = B.situ_moe_router(z, k, balance=True, packed=True, weights_dtype=F32)
    assert all(torch.equal(a, b) for a, b in zip(fresh, first))


@pytest.mark.parametrize("tokens", [20, 5000])
def test_router_graph(tokens):
    """A captured call is replayed on other logits, with eager calls between."""
    E, k = 200, 8
    g = gen_of(41)
    z = torch.randn(tokens, E, generator=g, device="cuda")
    dl = torch.tensor([2.0], device="cuda")
    dw = torch.randn(tokens, k, generator=g, device="cuda")

    def step():
        out = B.situ_moe_router(z, k, balance=True)
        return (*out, B.situ_moe_router_backward(z, out[0], dw, counts=out[2], d_loss=dl))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for i in range(4):
        z.copy_(torch.randn(tokens, E, generator=g, device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        want = step()
        assert all(torch.equal(a, b) for a, b in zip(held, want)), i


def test_router_streams():
    """Two calls at once on two streams, each with a workspace of its own."""
    g = gen_of(42)
    zs = [torch.randn(6000, 896, generator=g, device="cuda") for _ in range(2)]
    want = [B.situ_moe_router(z, 16, balance=True) for z in zs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in zs]
    for i in range(4):
        got = [B.situ_moe_router(z, 16, balance=True, stream=s) for z, s in zip(zs, streams)]
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert all(torch.equal(x, y) for x, y in zip(a, b)), i


def test_router_feeds_the_layer():
    """ids, weights and packed are what the layer's routing takes; -1 is outside every shard."""
    g = gen_of(43)
    T, E, k = 64, 40, 4
    z = torch.randn(T, E, generator=g, device="cuda")
    z[3, 2:] = NEG
    ids, weights, packed = B.situ_moe_router(z, k, packed=True)
    views = []
    for kw in (dict(topk_ids=ids, topk_weights=weights), dict(topk_packed=packed)):
        prob = B.make_problem(num_tokens=T, hidden_size=64, intermediate_size=32, num_experts=E, local_expert_offset=0,
                              local_num_experts=E, top_k=k, topk_packed="topk_packed" in kw)
        plan = B.situ_moe_plan(prob)
        ws = B.new_workspace(plan)
        ts = B.SituMoeTensors()
        for n, t in kw.items():
            setattr(ts, n, t.data_ptr())
        B.situ_moe_route(plan, ts, ws)
        views.append([B.workspace_view(plan, ws, r, torch.int32, (n,)).cpu().numpy().copy()
                      for r, n in (("counts", E), ("inv", T * k))])
    flat = ids.cpu().numpy().ravel()
    assert np.array_equal(views[0][0], np.bincount(flat[flat >= 0], minlength=E))
    assert np.array_equal(views[0][0], views[1][0]) and np.array_equal(views[0][1], views[1][1])
    assert np.array_equal(views[0][1] < 0, flat < 0)
