"""The gated activation, its 8-bit copy and its gradient against the formulas in
64 bits.

Tolerances.  u = 2^-24, m the largest of |g|, |a g|, |g / beta| and |u / lbeta| up to
100: an exponential's argument rounds twice, 3 m u relative in its value; tanh by
a quotient is within 6 u, by the exponential within 32 u of its value from 1/4
on; the products add some 20 u.  So a factor is within (6 m + 64) u, h and the
terms of a gradient within (12 m + 128) u of their magnitudes, before the one
rounding to bf16, 2^-8 of the value.  An exponential below fp32's smallest normal
value, 2^-126, may be taken for 0, and so may a product below it: at most 2^-126
times the product of the other factors, which is below 16 (1 + |g|) (1 + |u|) (1 + |dh|)
for the constants below 2.3 used here, twice or three times.  Codes and scales
are the quantization's.
"""

import numpy as np
import pytest
import torch

import block_scaled_mxfp4_amd as B

pytestmark = pytest.mark.gpu

BF, F32, D = torch.bfloat16, torch.float32, torch.float64
F8 = torch.float8_e4m3fn
U = 2.0 ** -24
KINDS = {"situ": ("situ_beta", "situ_linear_beta"), "swiglu": (), "swiglu_bias": ("swiglu_alpha", "swiglu_beta")}


def gen_of(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def offsets_of(counts):
    return torch.tensor([0] + list(np.cumsum(counts)), dtype=torch.int32, device="cuda")


def padded(t, pad):
    """The same rows with `pad` elements of NaN between them."""
    whole = torch.full((t.shape[0], t.shape[1] + pad), float("nan"), dtype=t.dtype, device="cuda")
    whole[:, :t.shape[1]] = t
    return whole[:, :t.shape[1]]


def constants(kind, g, experts):
    return {n: 0.3 + 2 * torch.rand(experts, generator=g, device="cuda") for n in KINDS[kind]}


def per_row(kind, con, counts):
    e = torch.repeat_interleave(torch.arange(len(counts), device="cuda"), torch.tensor(counts, device="cuda"))
    return [con[n].to(D)[e, None] for n in KINDS[kind]]


def formulas(kind, g, u, dh, p):
    """h, dg, du and the magnitudes dg adds; m of the tolerance."""
    s, left = torch.sigmoid(g), torch.sigmoid(-g)
    if kind == "situ":
        b, l = p
        e1, e2 = torch.exp(-2 * (g / b).abs()), torch.exp(-2 * (u / l).abs())
        t1, s1, t2, s2 = torch.tanh(g / b), 4 * e1 / (1 + e1) ** 2, torch.tanh(u / l), 4 * e2 / (1 + e2) ** 2
        gate, up = b * t1 * s, l * t2
        dg = dh * up * (s1 * s + gate * left)
        mag = (dh * up).abs() * (s1 * s + (gate * left).abs())
        return gate * up, dg, dh * gate * s2, mag, torch.stack([x.abs().expand_as(g) for x in (g, g / b, u / l)]).amax(0)
    a, c = p if p else (torch.ones((), dtype=D, device="cuda"), 0.0)
    s, left = torch.sigmoid(a * g), torch.sigmoid(-a * g)
    gate, up = g * s, u + c
    mag = (dh * up).abs() * s * (1 + (a * g * left).abs())
    return gate * up, dh * up * s * (1 + a * g * left), dh * gate, mag, torch.maximum(g.abs(), (a * g).abs())


def close(got, want, mag, m, factors):
    tol = (12 * m.clamp(max=100.0) + 128) * U * mag + 2.0 ** -120 * factors
    tol = tol * (1 + 2.0 ** -8) + 2.0 ** -8 * want.abs() + 2.0 ** -133
    bad = ~((got.to(D) - want).abs() <= tol)
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[0].tolist(), got[bad][0].item(), want[bad][0].item())


def quantized(gate_up, inner):
    """Codes and scales of the two halves by the quantization itself, halves widened to whole blocks."""
    codes, scales = [], []
    for half in (gate_up[:, :inner], gate_up[:, inner:]):
        wide = torch.zeros(half.shape[0], -(-inner // 128) * 128, dtype=BF, device="cuda")
        wide[:, :inner] = half
        c, s = B.situ_moe_quantize_fp8_block128(wide)
        codes.append(c[:, :inner])
        scales.append(s)
    return torch.cat(codes, 1), torch.cat(scales, 1)


def widened(codes, scales, inner):
    col = torch.arange(2 * inner, device="cuda")
    return codes.view(F8).to(D) * scales.to(D)[:, col // inner * -(-inner // 128) + col % inner // 128]


COUNTS = {"one_row": [1], "single": [0, 0, 1, 0], "ragged": [3, 0, 17, 64, 65, 0, 127, 1],
          "many": [(7 * i) % 5 for i in range(333)], "all": [0] * 500 + [777] + [0] * 523}


@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("which", list(COUNTS))
@pytest.mark.parametrize("inner,pad", [(8, 0), (72, 8), (128, 0), (200, 16), (384, 0), (1000, 0), (1536, 64)])
def test_activation(inner, pad, which, kind):
    counts = COUNTS[which]
    rows = sum(counts)
    g = gen_of(inner + rows)
    con = constants(kind, g, len(counts))
    off = offsets_of(counts)
    wide = torch.exp(1.5 * torch.randn(rows, 1, generator=g, device="cuda"))
    gate_up = padded((torch.randn(rows, 2 * inner, generator=g, device="cuda") * wide).to(BF), pad)
    dh = padded(torch.randn(rows, inner, generator=g, device="cuda").to(BF), pad)
    p = per_row(kind, con, counts)
    kw = dict(activation=kind, offsets=off, **con)

    def against(gu, got_h, got_d):
        gate, up = gu[:, :inner], gu[:, inner:]
        h, dg, du, mag, m = formulas(kind, gate, up, dh.to(D), p)
        factors = (1 + gate.abs()) * (1 + up.abs())
        if got_h is not None:
            close(got_h, h, h.abs(), m, factors)
        if got_d is not None:
            factors = factors * (1 + dh.to(D).abs())
            close(got_d[:, :inner], dg, mag, m, factors)
            close(got_d[:, inner:], du, du.abs(), m, factors)

    h = B.situ_moe_activation(gate_up, **kw)
    against(gate_up.to(D), h, None)
    h2, codes, scales = B.situ_moe_activation(gate_up, checkpoint=True, **kw)
    assert torch.equal(h2, h)
    want_codes, want_scales = quantized(gate_up, inner)
    assert torch.equal(codes, want_codes) and torch.equal(scales, want_scales)
    d, again = B.situ_moe_activation_backward(dh, gate_up, recompute=True, **kw)
    against(gate_up.to(D), again, d)
    assert torch.equal(B.situ_moe_activation_backward(dh, gate_up, **kw), d)
    d, again = B.situ_moe_activation_backward(dh, codes, scales, recompute=True, **kw)
    against(widened(codes, scales, inner), again, d)
    assert torch.equal(B.situ_moe_activation_backward(dh, codes.view(F8), scales, **kw), d)


def test_codes_are_the_quantizations():
    """Where I is a multiple of 128 the codes and scales are those of the whole rows' quantization."""
    g = gen_of(3)
    gate_up = torch.randn(77, 1536, generator=g, device="cuda").to(BF)
    _, codes, scales = B.situ_moe_activation(gate_up, activation="swiglu", checkpoint=True)
    want = B.situ_moe_quantize_fp8_block128(gate_up)
    assert torch.equal(codes, want[0]) and torch.equal(scales, want[1])


@pytest.mark.parametrize("kind", list(KINDS))
def test_rows_of_no_group_stay(kind):
    """Rows before the first and behind the last group are neither read nor written."""
    g = gen_of(4)
    inner, rows = 136, 50
    off = torch.tensor([5, 5, 20, 41], dtype=torch.int32, device="cuda")
    con = constants(kind, g, 3)
    kw = dict(activation=kind, offsets=off, **con)
    gate_up = torch.randn(rows, 2 * inner, generator=g, device="cuda").to(BF)
    dh = torch.randn(rows, inner, generator=g, device="cuda").to(BF)
    gate_up[:5] = gate_up[41:] = float("nan")
    out, h2 = torch.full((rows, inner), 7.0, dtype=BF, device="cuda"), torch.full((rows, inner), 7.0, dtype=BF, device="cuda")
    d = torch.full((rows, 2 * inner), 7.0, dtype=BF, device="cuda")
    codes = torch.full((rows, 2 * inner), 9, dtype=torch.uint8, device="cuda")
    scales = torch.full((rows, 4), 7.0, device="cuda")
    B.situ_moe_activation(gate_up, out=out, codes=codes, scales=scales, **kw)
    B.situ_moe_activation_backward(dh, codes, scales, out=d, h=h2, **kw)
    for t, v in ((out, 7), (h2, 7), (d, 7), (codes, 9), (scales, 7)):
        assert (t[:5] == v).all() and (t[41:] == v).all()
        assert torch.isfinite(t[5:41].float()).all()
    assert torch.equal(out[5:41], B.situ_moe_activation(gate_up[5:41].clone(), activation=kind,
                                                        offsets=(off - 5), **con))


@pytest.mark.parametrize("kind", list(KINDS))
def test_lowest_values(kind):
    """The type's largest magnitudes, as masks leave them: the formulas' limits, though products on the way overflow."""
    low = torch.finfo(BF).min
    con = {n: torch.tensor([1.7], device="cuda") for n in KINDS[kind]}
    vals = torch.tensor([low, -low, 1e20, -1e20, 2.0 ** 21, -2.0 ** 21, 1000.0, -1000.0], dtype=BF, device="cuda")
    g, u = torch.meshgrid(vals, torch.cat([vals, torch.tensor([0.0, 3.0, -0.5], dtype=BF, device="cuda")]), indexing="ij")
    g, u = (t.reshape(1, -1) for t in (g, u))                   # 88 columns
    h = B.situ_moe_activation(torch.cat([g, u], 1), activation=kind, **con)
    for dh in (1.0, -0.02, 0.0):
        d_h = torch.full_like(g, dh)
        d, again = B.situ_moe_activation_backward(d_h, torch.cat([g, u], 1), activation=kind, recompute=True, **con)
        p = [con[n].to(D) for n in KINDS[kind]]
        wh, wg, wu, *_ = formulas(kind, g.to(D), u.to(D), d_h.to(D), p)
        # exponentials are 0 here and tanh and the sigmoid 0 or 1 up to 6 u; 1000 c rounds u + c by u of it
        for got, want in ((h, wh), (again, wh), (d[:, :88], wg), (d[:, 88:], wu)):
            over = torch.isinf(want.to(F32).to(BF))
            assert torch.equal(got[over], want[over].to(F32).to(BF))
            assert ((got[~over].to(D) - want[~over]).abs() <= (2.0 ** -8 + 64 * U) * want[~over].abs()).all()


@pytest.mark.parametrize("kind", list(KINDS))
def test_not_finite(kind):
    """NaN and infinities stay in their element; large magnitudes saturate as the formulas do."""
    con = {n: torch.tensor([1.5], device="cuda") for n in KINDS[kind]}
    base = torch.randn(4, 512, generator=gen_of(6), device="cuda").to(BF)
    want = B.situ_moe_activation(base, activation=kind, **con)
    x = base.clone()
    x[0, 3], x[1, 256 + 5] = float("nan"), float("nan")
    x[2, 7], x[2, 256 + 9] = 1e30, -1e30
    x[3, 1] = -1e30
    got = B.situ_moe_activation(x, activation=kind, **con)
    assert torch.isnan(got[0, 3]) and torch.isnan(got[1, 5])
    changed = torch.zeros(4, 256, dtype=torch.bool, device="cuda")
    changed[0, 3] = changed[1, 5] = changed[2, 7] = changed[2, 9] = changed[3, 1] = True
    assert torch.equal(got[~changed], want[~changed]) and torch.isfinite(got[2:]).all() and got[3, 1] == 0
    dh = torch.ones(4, 256, dtype=BF, device="cuda")
    d = B.situ_moe_activation_backward(dh, x, activation=kind, **con)
    assert torch.isnan(d[0, 3]) and torch.isnan(d[1, 5]) and torch.isfinite(d[2:]).all()
    # 8 bits: a NaN is one code, an infinity takes its block along
    x[2, 100] = float("inf")
    _, codes, scales = B.situ_moe_activation(x, activation=kind, checkpoint=True, **con)
    v = codes.view(F8).float()
    assert torch.isnan(v[0, 3]) and torch.isfinite(v[0, 4:]).all() and torch.isinf(scales[2, 0]) and torch.isnan(v[2, :128]).all()


@pytest.mark.parametrize("kind", list(KINDS))
def test_gradient_by_differences(kind):
    g = gen_of(7)
    con = {n: torch.tensor([0.8], device="cuda") for n in KINDS[kind]}
    p = [con[n].to(D)[:, None] for n in KINDS[kind]]
    gate_up = (2 * torch.randn(3, 16, generator=g, device="cuda")).to(BF)
    dh = torch.randn(3, 8, generator=g, device="cuda").to(BF)
    d = B.situ_moe_activation_backward(dh, gate_up, activation=kind, **con)
    step = 1e-6
    for r in range(3):
        for c in range(16):
            v = []
            for sign in (1, -1):
                x = gate_up.to(D).clone()
                x[r, c] += sign * step
                v.append((formulas(kind, x[:, :8], x[:, 8:], dh.to(D), p)[0] * dh.to(D)).sum())
            want = float((v[0] - v[1]) / (2 * step))
            assert abs(d[r, c].item() - want) <= 2.0 ** -8 * abs(want) + 1e-6, (r, c)


def test_in_place_and_repeats():
    g = gen_of(8)
    rows, inner = 2050, 264
    gate_up = torch.randn(rows, 2 * inner, generator=g, device="cuda").to(BF)
    dh = torch.randn(rows, inner, generator=g, device="cuda").to(BF)
    d, h = B.situ_moe_activation_backward(dh, gate_up, activation="swiglu", recompute=True)
    for _ in range(3):
        again = B.situ_moe_activation_backward(dh, gate_up, activation="swiglu", recompute=True)
        assert torch.equal(again[0], d) and torch.equal(again[1], h)
    x, y = gate_up.clone(), dh.clone()
    B.situ_moe_activation_backward(y, x, activation="swiglu", out=x, h=y)
    assert torch.equal(x, d) and torch.equal(y, h)


def test_past_32_bits():
    """Rows that begin past 2^32 bytes."""
    rows, inner = 140_000, 8192
    gate_up = torch.zeros(rows, 2 * inner, dtype=BF, device="cuda")
    g = gen_of(9)
    for r in (0, 65535, 131071, rows - 1):
        gate_up[r] = torch.randn(2 * inner, generator=g, device="cuda").to(BF)
    pick = torch.tensor([0, 65535, 131071, rows - 1], device="cuda")
    h, codes, scales = B.situ_moe_activation(gate_up, activation="swiglu", checkpoint=True)
    few = B.situ_moe_activation(gate_up[pick], activation="swiglu", checkpoint=True)
    assert all(torch.equal(a[pick], b) for a, b in zip((h, codes, scales), few))
    dh = torch.ones(rows, inner, dtype=BF, device="cuda")
    d = B.situ_moe_activation_backward(dh, codes, scales, activation="swiglu", out=gate_up)
    assert torch.equal(d[pick], B.situ_moe_activation_backward(dh[pick], *few[1:], activation="swiglu"))


def test_graph_and_streams():
    g = gen_of(10)
    rows, inner, counts = 300, 384, [100, 0, 150, 50]
    off = offsets_of(counts)
    con = constants("situ", g, 4)
    gate_up = torch.randn(rows, 2 * inner, generator=g, device="cuda").to(BF)
    dh = torch.randn(rows, inner, generator=g, device="cuda").to(BF)

    def step(**kw):
        h, codes, scales = B.situ_moe_activation(gate_up, offsets=off, checkpoint=True, **con, **kw)
        return (h, *B.situ_moe_activation_backward(dh, codes, scales, offsets=off, recompute=True, **con, **kw))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for i in range(4):
        gate_up.copy_(torch.randn(rows, 2 * inner, generator=g, device="cuda"))
        off.copy_(offsets_of([[300, 0, 0, 0], [0, 0, 0, 300], [1, 2, 3, 294], [75] * 4][i]))
        graph.replay()
        torch.cuda.synchronize()
        want = step()
        assert all(torch.equal(a, b) for a, b in zip(held, want)), i
        got = step(stream=side.cuda_stream)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want)), i
