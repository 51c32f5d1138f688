"""Adapters of many requests beside a shared projection against the formula in 64
bits.

Tolerances.  u = 2^-24.  The matrix instructions stay within 1.5 ulps of the
magnitudes they add per 32 products, so with M = |c| |b| (|a| |x|), the magnitudes
of the two products, the first is off by (8 + 1.5 k / 32) 2 u M and the second, with
its two terms, by (8 + 3 rank / 32) 2 u M; the two bf16 terms lose 2^-16 of M;
scale, parts and base add 20 roundings of what they add.  bf16 is rounded once
more, 2^-8 of the value.
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


def randn(g, *shape, dtype=BF, scale=1.0, pad=0):
    whole = torch.full(shape[:-1] + (shape[-1] + pad,), float("nan"), device="cuda")
    whole[..., :shape[-1]] = scale * torch.randn(shape, generator=g, device="cuda")
    return whole.to(dtype)[..., :shape[-1]]


def offsets_of(counts, first=0):
    return torch.tensor([first] + list(first + np.cumsum(counts)), dtype=torch.int32, device="cuda")


def check(x, a, b, offsets, adapter, base=None, ranks=None, scales=None, before=None, **kw):
    """The call against 64 bits; `before`: what rows of no request hold."""
    rows, k = x.shape
    held, rank, _ = a.shape
    n = b.shape[1]
    got = B.situ_moe_adapters(x, a, b, offsets, adapter, base=base, ranks=ranks, scales=scales, **kw)
    want = torch.zeros(rows, n, dtype=D, device="cuda") if base is None else base.to(D).clone()
    mag = torch.zeros(rows, n, dtype=D, device="cuda")
    bounds = offsets.tolist()
    own = torch.zeros(rows, dtype=torch.bool, device="cuda")
    for q, i in enumerate(adapter.tolist()):
        lo, hi = bounds[q], bounds[q + 1]
        own[lo:hi] = True
        if hi > lo and 0 <= i < held:
            r = rank if ranks is None else min(max(int(ranks[i]), 0), rank)
            c = 1.0 if scales is None else float(scales[i])
            xs, aa, bb = x[lo:hi].to(D), a[i, :r].to(D), b[i, :, :r].to(D)
            want[lo:hi] += c * (xs @ aa.t()) @ bb.t()
            mag[lo:hi] += abs(c) * (xs.abs() @ aa.abs().t()) @ bb.abs().t()
    tol = ((32 + 1.5 * k / 32 + 3 * rank / 32) * 2 * U + 2.0 ** -16) * mag + 20 * U * (want.abs() + mag) + 2.0 ** -120
    if got.dtype == BF:
        tol = tol * (1 + 2.0 ** -8) + 2.0 ** -8 * want.abs() + 2.0 ** -133
    bad = ~((got.to(D) - want).abs() <= tol) & own[:, None]
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[0].tolist(), got[bad][0].item(), want[bad][0].item())
    if before is not None:
        assert (got[~own] == before).all()
    return got


SHAPES = [(8, 8, 8), (64, 128, 16), (264, 200, 16), (1000, 72, 32), (520, 3584, 24), (136, 1040, 64), (72, 264, 128),
          (200, 136, 256), (136, 8200, 24), (264, 2056, 72)]                   # n, k, rank
BATCHES = {"one_token": [1], "decode": [1] * 37, "decode_large": [1] * 131, "ragged": [3, 0, 17, 1, 64, 0, 0, 33, 2],
           "long": [300, 0, 5, 411], "many_empty": [0] * 150 + [5] + [0] * 200 + [40, 1] + [0] * 90,
           "many": [(5 * i) % 4 for i in range(700)]}


@pytest.mark.parametrize("n,k,rank", SHAPES)
@pytest.mark.parametrize("batch", list(BATCHES))
def test_adapters(batch, n, k, rank):
    counts = BATCHES[batch]
    rows, held = sum(counts), 7
    g = gen_of(n + k + rows)
    rng = np.random.RandomState(n + rows)
    offsets = offsets_of(counts)
    adapter = torch.from_numpy(rng.randint(-1, held + 1, len(counts)).astype(np.int32)).cuda()   # -1 and `held`: none
    a, b = randn(g, held, rank, k, scale=k ** -0.5), randn(g, held, n, rank, scale=rank ** -0.5)
    x = randn(g, rows, k, pad=8)
    scales = torch.randn(held, generator=g, device="cuda")
    for dtype in (BF, F32):
        base = randn(g, rows, n, dtype=dtype, pad=16)
        got = check(x, a, b, offsets, adapter, base, scales=scales)
        assert got.dtype == dtype
        none = (adapter < 0) | (adapter >= held)
        rowless = torch.repeat_interleave(none, offsets.diff().long())
        assert torch.equal(got[rowless], base[rowless])
        assert torch.equal(B.situ_moe_adapters(x, a, b, offsets, adapter, base=base, scales=scales), got)
        inplace = base.clone()
        assert B.situ_moe_adapters(x, a, b, offsets, adapter, base=inplace, scales=scales, out=inplace) is inplace
        assert torch.equal(inplace, got)
    check(x, a, b, offsets, adapter)
    ranks = torch.tensor([0, rank, 3, rank + 5, -2, 8, rank - 1], dtype=torch.int32, device="cuda")
    an, bn = a.clone(), b.clone()
    for i, r in enumerate(ranks.tolist()):              # what lies past an adapter's rank may be anything
        an[i, max(r, 0):] = float("nan")
        bn[i, :, max(r, 0):] = float("inf")
    check(x, an, bn, offsets, adapter, base, ranks=ranks, out_dtype=F32)


def test_rows_of_no_request_stay():
    g = gen_of(2)
    for rows, first, counts in ((50, 5, [10, 0, 20]), (600, 40, [100, 300]), (64, 0, [0, 0])):
        x, base = randn(g, rows, 64), randn(g, rows, 128)
        x[:first] = float("nan")
        a, b = randn(g, 3, 16, 64), randn(g, 3, 128, 16)
        offsets = offsets_of(counts, first)
        adapter = torch.arange(len(counts), dtype=torch.int32, device="cuda")
        out = torch.full((rows, 128), 9.0, dtype=BF, device="cuda")
        check(x, a, b, offsets, adapter, base, before=9.0, out=out)


@pytest.mark.parametrize("counts", [[1] * 20, [5, 9, 30, 3], [100, 200, 300]])
def test_requests_keep_to_themselves(counts):
    """NaN and infinities in one request's rows, adapter or scale do not reach another's rows in the same tile."""
    g = gen_of(3)
    rows = sum(counts)
    x, base = randn(g, rows, 200), randn(g, rows, 136)
    held = len(counts) + 1
    a, b = randn(g, held, 16, 200), randn(g, held, 136, 16)
    scales = torch.ones(held, device="cuda")
    offsets = offsets_of(counts)
    adapter = torch.arange(len(counts), dtype=torch.int32, device="cuda")
    want = B.situ_moe_adapters(x, a, b, offsets, adapter, base=base, scales=scales)
    a[1], b[2], scales[3] = float("nan"), float("inf"), float("inf")
    x[0] = float("nan")
    got = B.situ_moe_adapters(x, a, b, offsets, adapter, base=base, scales=scales)
    keep = torch.ones(rows, dtype=torch.bool, device="cuda")
    keep[offsets[1]:offsets[min(4, len(counts))]] = False
    keep[0] = False
    assert torch.equal(got[keep], want[keep])
    assert torch.isnan(got[0]).all() and torch.isnan(got[offsets[1]:offsets[2]]).all()


def test_large_values():
    """Between the products t may be large: two terms of an infinity are one."""
    x = torch.full((3, 64), 2.0 ** 60, dtype=BF, device="cuda")
    a = torch.full((1, 8, 64), 2.0 ** 66, dtype=BF, device="cuda")
    b = torch.full((1, 8, 8), 2.0 ** -80, dtype=BF, device="cuda")
    off, ids = offsets_of([3]), torch.zeros(1, dtype=torch.int32, device="cuda")
    assert torch.isinf(B.situ_moe_adapters(x, a, b, off, ids)).all()
    a[:] = 2.0 ** 50
    check(x, a, b, off, ids)


def test_as_the_grouped_products():
    """One request per adapter: the two grouped products give the same adapter."""
    g = gen_of(4)
    counts = [40, 0, 90, 7]
    off = offsets_of(counts)
    rows, k, n, r = sum(counts), 512, 264, 16
    x = randn(g, rows, k)
    a, b = randn(g, 4, r, k, scale=k ** -0.5), randn(g, 4, n, r, scale=r ** -0.5)
    got = check(x, a, b, off, torch.arange(4, dtype=torch.int32, device="cuda"), out_dtype=F32)
    t = B.situ_moe_grouped_matmul(x, a, off)
    want = B.situ_moe_grouped_matmul(t, b, off, out_dtype=F32)
    mag = torch.zeros_like(got)
    for i, (lo, hi) in enumerate(zip(off.tolist()[:-1], off.tolist()[1:])):
        mag[lo:hi] = (x[lo:hi].float().abs() @ a[i].float().abs().t()) @ b[i].float().abs().t()
    assert ((got - want).abs() <= 2.0 ** -8 * mag).all()       # the grouped products round t to bf16


def test_beside_the_fp8_projection():
    """Adapters added to the FP8 projection they stand beside, in place."""
    g = gen_of(5)
    rows, k, n = 20, 512, 384
    x, w = randn(g, rows, k), randn(g, n, k, scale=k ** -0.5)
    w8 = torch.empty(n, k, dtype=torch.uint8, device="cuda")
    ws = torch.empty(n // 128, k // 128, device="cuda")
    for i in range(n // 128):
        for j in range(k // 128):
            blk = w[128 * i:128 * (i + 1), 128 * j:128 * (j + 1)].float()
            ws[i, j] = blk.abs().max() / 448
            w8[128 * i:128 * (i + 1), 128 * j:128 * (j + 1)] = (blk / ws[i, j]).to(torch.float8_e4m3fn).view(torch.uint8)
    y = B.situ_moe_matmul_fp8_block128(*B.situ_moe_quantize_fp8_block128(x), w8, ws)
    a, b = randn(g, 5, 16, k, scale=k ** -0.5), randn(g, 5, n, 16, scale=0.25)
    off = offsets_of([1] * 10 + [10])
    ids = torch.tensor([0, 1, 2, 3, 4, -1, 0, 1, 2, 3, 4], dtype=torch.int32, device="cuda")
    before = y.clone()
    want = check(x, a, b, off, ids, before)
    assert torch.equal(B.situ_moe_adapters(x, a, b, off, ids, base=y, out=y), want)


def test_past_32_bits():
    rows, k, n = 310_000, 7168, 64
    g = gen_of(6)
    x = torch.zeros(rows, k, dtype=BF, device="cuda")
    x[-40:] = torch.randn(40, k, generator=g, device="cuda").to(BF)
    a, b = randn(g, 2, 16, k, scale=k ** -0.5), randn(g, 2, n, 16)
    off = torch.tensor([0, rows - 30, rows], dtype=torch.int32, device="cuda")
    ids = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    got = B.situ_moe_adapters(x, a, b, off, ids, out_dtype=F32)
    few = B.situ_moe_adapters(x[-40:].clone(), a, b, torch.tensor([0, 10, 40], dtype=torch.int32, device="cuda"), ids, out_dtype=F32)
    t = x[-40:].float().abs().max() * a.float().abs().max() * k * 16 * b.float().abs().max()
    assert (got[-40:] - few).abs().max() <= 1e-5 * t and not got[:-40].any()
    wide = torch.zeros(rows, 7168, dtype=BF, device="cuda")       # out past 2^32 bytes
    b = randn(g, 2, 7168, 16)
    B.situ_moe_adapters(x, a, b, off, ids, base=wide, out=wide)
    few = check(x[-40:].clone(), a, b, torch.tensor([0, 10, 40], dtype=torch.int32, device="cuda"), ids)
    assert ((wide[-40:].float() - few.float()).abs() <= 2.0 ** -7 * few.float().abs() + 1e-5 * t).all() and not wide[:-40].any()


def test_graph_and_streams():
    g = gen_of(7)
    rows, k, n, held = 48, 1024, 520, 6
    x, base = randn(g, rows, k), randn(g, rows, n)
    a, b = randn(g, held, 16, k, scale=k ** -0.5), randn(g, held, n, 16)
    off, ids = offsets_of([1] * 40 + [8]), torch.zeros(41, dtype=torch.int32, device="cuda")

    def step(**kw):
        return B.situ_moe_adapters(x, a, b, off, ids, base=base, **kw)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held_out = step()
    for i in range(4):
        ids.copy_(torch.randint(-1, held, (41,), generator=g, device="cuda"))
        off.copy_(offsets_of([[1] * 40 + [8], [0] * 40 + [48], [48] + [0] * 40, [2] * 20 + [0] * 20 + [8]][i]))
        x.copy_(randn(g, rows, k))
        graph.replay()
        torch.cuda.synchronize()
        want = step()
        got = step(stream=side)
        torch.cuda.synchronize()
        assert torch.equal(held_out, want) and torch.equal(got, want), i
