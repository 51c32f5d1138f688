"""FP8 products with scales per 128 and bf16 products grouped by expert, with
their gradients, against the same formulas in 64 bits.

Tolerances.  u = 2^-24.  An fp32 output is the kernel's sum: the matrix-core
instructions stay within 1.5 ulps of the magnitudes they add per 32 products
(the bound of gpu_helpers.acc_error_ulps), so K products are off by at most
(8 + 1.5 K / 32) 2 u times S, the sum of the products' magnitudes; the FP8
product adds two roundings per 128 (the scales' product and the fused
multiply-add): 2 ulps per 32 covers both.  A bf16 output is that rounded once:
half a step, 2^-8 of the value, more.

FP8 products with a bf16 output run on the FP8 matrix-core instruction.  It
adds the eight products of each aligned eight elements of k in fixed point and
drops what lies 13 bits below the leading bit of the largest (measured on
gfx950 with two addends, every position and distance).  A product's own bits
span 8, so the largest loses nothing, and each of the seven others less than
2^-13 of it: 7 * 2^-13 of the largest product of each eight, G in all, is
added to the tolerance.
"""

import numpy as np
import pytest
import torch

import block_scaled_mxfp4_amd as B
import synthetic as S

pytestmark = pytest.mark.gpu

F8 = torch.float8_e4m3fn
BF, F32 = torch.bfloat16, torch.float32
D = torch.float64


def close(got, want, mag, K, per32=1.5, eights=None):
    """Every element of got within the tolerance of want; mag: S of each element, eights: G."""
    assert got.shape == want.shape
    tol = (8 + per32 * K / 32) * 2.0 ** -23 * mag
    if got.dtype == BF:
        if eights is not None:
            tol = tol + 7 * 2.0 ** -13 * eights
        tol = tol * (1 + 2.0 ** -8) + 2.0 ** -8 * want.abs() + 2.0 ** -133   # half of bf16's smallest step
    err = (got.to(D) - want).abs()
    bad = ~(err <= tol)
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[0].tolist(), err[bad][0].item(), tol[bad][0].item())


def offsets_of(counts):
    return torch.tensor([0] + list(np.cumsum(counts)), dtype=torch.int32, device="cuda")


def randn(gen, *shape, dtype=BF, pad=0):
    """Normal values; pad: elements between the rows that belong to nobody, set to NaN."""
    t = torch.full(shape[:-1] + (shape[-1] + pad,), float("nan"), device="cuda")
    t[..., :shape[-1]] = torch.randn(shape, generator=gen, device="cuda")
    return t.to(dtype)[..., :shape[-1]]


def gen_of(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


COUNTS = {
    "one_row": [1],
    "single": [0, 0, 1, 0],
    "ragged": [3, 0, 17, 64, 65, 0, 127, 1],
    "long": [300, 0, 5],
    "many": [(7 * i) % 5 for i in range(333)],
}

# (n, k): ranks on either side, sizes around the tiles' and steps' edges, odd n (the forward product)
SIZES = [(8, 8), (16, 264), (264, 16), (40, 72), (128, 64), (136, 520), (200, 328), (64, 1024)]


# ----------------------------------------------------------------- quantize

def quant64(x):
    rows, cols = x.shape
    f = torch.nn.functional.pad(x.to(D), (0, -cols % 128)).view(rows, -1, 128)
    scale = f.abs().amax(2).clamp(min=2.0 ** -100) / 448
    return (f / scale[..., None]).view(rows, -1)[:, :cols], scale


@pytest.mark.parametrize("rows,cols,pad", [(1, 16, 0), (1, 128, 0), (5, 144, 16), (33, 3584, 0), (64, 7168, 8),
                                           (1000, 272, 48), (4099, 1024, 0)])
def test_quantize(rows, cols, pad):
    g = gen_of(rows + cols)
    x = (randn(g, rows, cols, dtype=F32, pad=pad) *
         torch.exp(4 * torch.randn(rows, 1, generator=g, device="cuda"))).to(BF)
    if pad:
        whole = torch.full((rows, cols + pad), float("nan"), dtype=BF, device="cuda")
        whole[:, :cols] = x
        x = whole[:, :cols]
    x[0, :16] = 0
    if rows > 2:
        x[1] = 0                                    # blocks of zeros
        x[2] *= 2.0 ** -110                         # blocks below the scale's floor
    codes, scales = B.situ_moe_quantize_fp8_block128(x)
    q, want = quant64(x)
    assert codes.dtype == torch.uint8 and scales.shape == want.shape
    # the division by 448 rounds once
    assert ((scales.to(D) - want).abs() <= 2.0 ** -24 * want).all()
    v = codes.view(F8).to(D)
    # half an E4M3 step (2^-4 of the value, 2^-10 below 2^-6) of the quotient by the rounded scale
    qs = x.to(D) / scales.to(D).repeat_interleave(128, 1)[:, :cols]
    assert ((v - qs).abs() <= torch.clamp(2.0 ** -4 * qs.abs(), min=2.0 ** -10) * (1 + 2.0 ** -20)).all()
    # and it is the nearest value: torch's own cast of the fp32 quotient
    near = (x.float() / scales.repeat_interleave(128, 1)[:, :cols]).to(F8).float()
    assert torch.equal(v.float(), near)
    assert torch.isfinite(v).all()


def test_quantize_many_rows():
    x = torch.randn(1 << 19, 640, device="cuda").to(BF)      # more blocks than the grid has workgroups for at once
    codes, scales = B.situ_moe_quantize_fp8_block128(x)
    want = x.view(-1, 5, 128).abs().amax(2).float() / 448
    assert ((scales - want).abs() <= 2.0 ** -23 * want).all()
    near = (x.float() / scales.repeat_interleave(128, 1)).to(F8)
    assert torch.equal(codes, near.view(torch.uint8))


def test_quantize_not_finite():
    x = torch.randn(3, 256, device="cuda").to(BF)
    x[0, 5] = float("nan")
    x[1, 200] = float("inf")
    x[2, 10] = -float("inf")
    codes, scales = B.situ_moe_quantize_fp8_block128(x)
    v = codes.view(F8).float()
    assert torch.isnan(v[0, 5]) and torch.isfinite(v[0, :5]).all() and torch.isfinite(v[0, 6:]).all()
    assert torch.isfinite(scales[0]).all()
    assert torch.isnan(v[1, 128:]).all() and torch.isfinite(v[1, :128]).all() and torch.isinf(scales[1, 1])
    assert torch.isnan(v[2, :128]).all() and torch.isfinite(v[2, 128:]).all() and torch.isinf(scales[2, 0])


# ---------------------------------------------------------------- FP8 product

def fp8_inputs(g, rows, experts, n, k, pad=0):
    kb, nb = -(-k // 128), -(-n // 128)
    a = torch.randint(0, 256, (rows, k + pad), generator=g, device="cuda", dtype=torch.uint8)
    w = torch.randint(0, 256, (experts, n, k), generator=g, device="cuda", dtype=torch.uint8)
    for t in (a, w):
        t[(t & 0x7f) == 0x7f] = 0x3c                # no NaN codes
    if pad:
        a[:, k:] = 0x7f
    sa = torch.rand(rows, kb, generator=g, device="cuda") + 0.01
    sw = torch.rand(experts, nb, kb, generator=g, device="cuda") - 0.5
    return a[:, :k], sa, w, sw


def fp8_ref(a, sa, w, sw, counts):
    rows, k = a.shape
    n = w.shape[1]
    a64 = a.contiguous().view(F8).to(D) * sa[:rows].to(D).repeat_interleave(128, 1)[:, :k]
    out, mag, eights, lo = [], [], [], 0
    for e, c in enumerate(counts):
        w64 = w[e].view(F8).to(D) * sw[e].to(D).repeat_interleave(128, 0)[:n].repeat_interleave(128, 1)[:, :k]
        out.append(a64[lo:lo + c] @ w64.t())
        mag.append(a64[lo:lo + c].abs() @ w64.abs().t())
        g = torch.zeros(c, n, dtype=D, device="cuda")
        for q in range(0, k, 8) if c else ():
            p = a64[lo:lo + c, None, q:q + 8].abs() * w64[None, :, q:q + 8].abs() if c * n < 1 << 21 else \
                a64[lo:lo + c, q:q + 8].abs().amax(1)[:, None, None] * w64[:, q:q + 8].abs().amax(1)[None, :, None]
            g += p.amax(2)
        eights.append(g)
        lo += c
    return torch.cat(out), torch.cat(mag), torch.cat(eights)


@pytest.mark.parametrize("rows,n,k,pad,out", [
    (1, 1, 16, 0, F32), (1, 128, 128, 0, BF), (1, 3584, 3584, 0, BF), (2, 129, 144, 16, F32), (16, 64, 256, 0, BF),
    (17, 200, 1040, 0, F32), (45, 1000, 912, 48, BF), (64, 384, 512, 0, BF), (130, 259, 400, 0, BF),
    (257, 513, 128, 0, F32), (300, 256, 2048, 128, BF), (1025, 640, 272, 0, BF), (2100, 2304, 1152, 0, BF)])
def test_fp8_dense(rows, n, k, pad, out):
    g = gen_of(rows * 7 + n)
    a, sa, w, sw = fp8_inputs(g, rows, 1, n, k, pad)
    got = B.situ_moe_matmul_fp8_block128(a, sa, w[0], sw[0], out_dtype=out)
    want, mag, eights = fp8_ref(a, sa, w, sw, [rows])
    close(got, want, mag, k, 2.0, eights)


@pytest.mark.parametrize("counts", COUNTS)
@pytest.mark.parametrize("n,k,out", [(1, 16, BF), (72, 400, F32), (256, 256, BF), (300, 1152, BF)])
def test_fp8_grouped(counts, n, k, out):
    c = COUNTS[counts]
    g = gen_of(n + len(c))
    rows = sum(c) + 3
    a, sa, w, sw = fp8_inputs(g, rows, len(c), n, k)
    a[sum(c):] = 0x7f                               # rows of no group, and experts without rows: NaN
    for e in range(len(c)):
        if c[e] == 0:
            w[e] = 0x7f
    got = torch.full((rows, n + 5), 3.0, dtype=out, device="cuda")
    B.situ_moe_matmul_fp8_block128(a, sa, w, sw, offsets=offsets_of(c), out=got[:, :n])
    want, mag, eights = fp8_ref(a[:sum(c)], sa, w, sw, c)
    close(got[:sum(c), :n], want, mag, k, 2.0, eights)
    assert (got[sum(c):] == 3.0).all() and (got[:, n:] == 3.0).all()


def test_fp8_scales_alone():
    """Codes of one and a scale of its own per block: the sum of the scales' products."""
    rows, n, k = 70, 400, 640
    a = torch.full((rows, k), 0x38, dtype=torch.uint8, device="cuda")
    w = torch.full((n, k), 0x38, dtype=torch.uint8, device="cuda")
    sa = torch.arange(rows * 5, device="cuda", dtype=F32).view(rows, 5) + 1
    sw = torch.arange(4 * 5, device="cuda", dtype=F32).view(4, 5) + 1
    got = B.situ_moe_matmul_fp8_block128(a, sa, w, sw, out_dtype=F32)
    want = 128 * (sa.to(D) @ sw.to(D).t()).repeat_interleave(128, 1)[:, :n]
    assert torch.equal(got.to(D), want)             # integers below 2^24


# ------------------------------------------------------------ grouped products

def grouped_ref(x, w, counts):
    out, mag, lo = [], [], 0
    for e, c in enumerate(counts):
        xe, we = x[lo:lo + c].to(D), w[e].to(D)
        out.append(xe @ we.t())
        mag.append(xe.abs() @ we.abs().t())
        lo += c
    return torch.cat(out), torch.cat(mag)


@pytest.mark.parametrize("counts", COUNTS)
@pytest.mark.parametrize("n,k", SIZES + [(1, 8), (77, 136)])
def test_forward(counts, n, k):
    c = COUNTS[counts]
    g = gen_of(n * 31 + k)
    rows = sum(c) + 2
    out = BF if n % 16 else F32
    x, w = randn(g, rows, k, pad=8), randn(g, len(c), n, k)
    x[sum(c):] = float("nan")
    for e in range(len(c)):
        if c[e] == 0:
            w[e] = float("nan")
    got = torch.full((rows, n + 3), 3.0, dtype=out, device="cuda")
    B.situ_moe_grouped_matmul(x, w, offsets_of(c), out=got[:, :n])
    want, mag = grouped_ref(x[:sum(c)], w, c)
    close(got[:sum(c), :n], want, mag, k)
    assert (got[sum(c):] == 3.0).all() and (got[:, n:] == 3.0).all()


@pytest.mark.parametrize("counts", COUNTS)
@pytest.mark.parametrize("n,k", SIZES)
def test_gradients(counts, n, k):
    c = COUNTS[counts]
    g = gen_of(n * 17 + k)
    rows = sum(c) + 2
    x, w, dy = randn(g, rows, k, pad=16), randn(g, len(c), n, k), randn(g, rows, n, pad=8)
    x[sum(c):] = float("nan")
    dy[sum(c):] = float("inf")
    dx = torch.full((rows, k), 3.0, dtype=BF if k % 16 else F32, device="cuda")
    B.situ_moe_grouped_matmul_dgrad(dy, w, offsets_of(c), out=dx)
    want, mag = grouped_ref(dy[:sum(c)], w.transpose(1, 2), c)
    close(dx[:sum(c)], want, mag, n)
    assert (dx[sum(c):] == 3.0).all()
    for out in (F32, BF):
        dw = B.situ_moe_grouped_matmul_wgrad(dy, x, offsets_of(c), out_dtype=out)
        lo = 0
        for e, m in enumerate(c):
            xe, de = x[lo:lo + m].to(D), dy[lo:lo + m].to(D)
            close(dw[e], de.t() @ xe, de.abs().t() @ xe.abs(), m)
            lo += m


def test_gradients_by_differences():
    """A step along one direction of x and one of w changes sum(out * dy) by the gradients' products with it."""
    c, n, k = [5, 0, 70, 33], 48, 72
    g = gen_of(5)
    rows = sum(c)
    x, w, dy = randn(g, rows, k), randn(g, len(c), n, k), randn(g, rows, n)
    off = offsets_of(c)
    dx = B.situ_moe_grouped_matmul_dgrad(dy, w, off, out_dtype=F32).to(D)
    dw = B.situ_moe_grouped_matmul_wgrad(dy, x, off).to(D)
    loss = lambda a, b: (B.situ_moe_grouped_matmul(a, b, off, out_dtype=F32).to(D) * dy.to(D)).sum().item()  # noqa: E731
    # the product is linear in each operand: a difference of any length is exact but for the sums' rounding
    vx, vw = randn(g, rows, k), randn(g, len(c), n, k)
    scale = (dx.abs() * vx.to(D).abs()).sum().item()
    x2 = (x.float() + vx.float()).to(BF)
    assert abs(loss(x2, w) - loss(x, w) - (dx * (x2.to(D) - x.to(D))).sum().item()) <= 1e-4 * scale
    w2 = (w.float() + vw.float()).to(BF)
    scale = (dw.abs() * vw.to(D).abs()).sum().item()
    assert abs(loss(x, w2) - loss(x, w) - (dw * (w2.to(D) - w.to(D))).sum().item()) <= 1e-4 * scale


@pytest.mark.parametrize("top_k", [1, 3, 16])
@pytest.mark.parametrize("n,k", [(16, 264), (264, 16), (136, 72)])
def test_pairs(top_k, n, k):
    c = [0, 40, 1, 0, 90, 29]
    rows, tokens = sum(c), -(-sum(c) * 2 // top_k)
    g = gen_of(top_k)
    pairs = torch.randperm(tokens * top_k, generator=g, device="cuda")[:rows].to(torch.int32)
    off = offsets_of(c)
    xt, w, dyp = randn(g, tokens, k), randn(g, len(c), n, k), randn(g, tokens * top_k, n, pad=8)
    x = xt[pairs.long() // top_k]
    # forward: token rows in, pair rows out
    got = torch.full((tokens * top_k, n), 3.0, dtype=BF, device="cuda")
    B.situ_moe_grouped_matmul(xt, w, off, pairs=pairs, x_div=top_k, out_div=1, out=got)
    want, mag = grouped_ref(x, w, c)
    close(got[pairs.long()], want, mag, k)
    rest = torch.ones(tokens * top_k, dtype=torch.bool, device="cuda")
    rest[pairs.long()] = False
    assert (got[rest] == 3.0).all()
    # dx: pair rows in, pair rows out
    dy = dyp[pairs.long()]
    dx = torch.full((tokens * top_k, k), 3.0, dtype=F32, device="cuda")
    B.situ_moe_grouped_matmul_dgrad(dyp, w, off, pairs=pairs, dy_div=1, out_div=1, out=dx)
    want, mag = grouped_ref(dy, w.transpose(1, 2), c)
    close(dx[pairs.long()], want, mag, n)
    assert (dx[rest] == 3.0).all()
    # dw: both gathered, or one
    for a, b, kw in ((dyp, xt, dict(dy_div=1, x_div=top_k)), (dy, xt, dict(x_div=top_k)), (dyp, x, dict(dy_div=1))):
        dw = B.situ_moe_grouped_matmul_wgrad(a, b, off, pairs=pairs, **kw)
        lo = 0
        for e, m in enumerate(c):
            xe, de = x[lo:lo + m].to(D), dy[lo:lo + m].to(D)
            close(dw[e], de.t() @ xe, de.abs().t() @ xe.abs(), m)
            lo += m


def test_long_contraction_and_many_rows():
    g = gen_of(3)
    n, k, rows = 72, 4104, 9001
    x, w, dy = randn(g, rows, k), randn(g, 2, n, k), randn(g, rows, n)
    c = [9000, 1]
    want, mag = grouped_ref(x, w, c)
    close(B.situ_moe_grouped_matmul(x, w, offsets_of(c), out_dtype=F32), want, mag, k)
    dw = B.situ_moe_grouped_matmul_wgrad(dy, x, offsets_of(c))
    close(dw[0], dy[:9000].to(D).t() @ x[:9000].to(D), dy[:9000].to(D).abs().t() @ x[:9000].to(D).abs(), 9000)
    # dense: no offsets
    want, mag = grouped_ref(x, w[:1], [rows])
    close(B.situ_moe_grouped_matmul(x, w[:1].contiguous()), want, mag, k)


# sizes at which each tile shape is taken, with rows, columns and contractions that end inside tiles
LARGE = {
    "pair": ([3000, 0, 2500, 1, 3499], 4104, 1096),
    "large": ([2050], 3592, 520),
    "split": ([60, 0, 45], 520, 1800),
    "split2": ([130], 8200, 1032),
    "short": ([700, 33, 0, 290], 784, 104),
    "thin": ([700, 33, 0, 290], 784, 40),
}


@pytest.mark.parametrize("shape", LARGE)
@pytest.mark.parametrize("out", [BF, F32])
def test_tile_shapes(shape, out):
    c, n, k = LARGE[shape]
    g = gen_of(len(shape))
    rows, off = sum(c), offsets_of(c)
    x, w = randn(g, rows, k), randn(g, len(c), n, k)
    want, mag = grouped_ref(x, w, c)
    close(B.situ_moe_grouped_matmul(x, w, off, out_dtype=out), want, mag, k)
    # dx of the transposed sizes: contraction k, columns n
    wt = w.transpose(1, 2).contiguous()
    close(B.situ_moe_grouped_matmul_dgrad(x, wt, off, out_dtype=out), want, mag, k)
    if k % 16 == 0 or shape == "pair":
        k8 = k // 16 * 16
        a, sa, w8, sw = fp8_inputs(g, rows, len(c), n - 5, k8)
        want, mag, eights = fp8_ref(a, sa, w8, sw, c)
        close(B.situ_moe_matmul_fp8_block128(a, sa, w8, sw, offsets=off, out_dtype=out), want, mag, k8, 2.0, eights)


@pytest.mark.parametrize("rows,experts,n,k", [(60, 16, 136, 520), (700, 40, 264, 40), (700, 40, 264, 104),
                                              (900, 8, 520, 1032), (9000, 6, 2056, 1032)])
def test_all_rows_in_one_group(rows, experts, n, k):
    """The shapes are chosen by the mean; a group may hold all rows."""
    g = gen_of(rows + n)
    c = [0] * (experts - 2) + [rows, 0]
    off = offsets_of(c)
    x, w, dy = randn(g, rows, k), randn(g, experts, n, k), randn(g, rows, n)
    want, mag = grouped_ref(x, w, c)
    close(B.situ_moe_grouped_matmul(x, w, off), want, mag, k)
    want, mag = grouped_ref(dy, w.transpose(1, 2), c)
    close(B.situ_moe_grouped_matmul_dgrad(dy, w, off), want, mag, n)
    dw = B.situ_moe_grouped_matmul_wgrad(dy, x, off)
    close(dw[-2], dy.to(D).t() @ x.to(D), dy.to(D).abs().t() @ x.to(D).abs(), rows)
    assert (dw[:-2] == 0).all() and (dw[-1] == 0).all()
    a, sa, w8, sw = fp8_inputs(g, rows, experts, n, k // 16 * 16)
    want, mag, eights = fp8_ref(a, sa, w8, sw, c)
    close(B.situ_moe_matmul_fp8_block128(a, sa, w8, sw, offsets=off), want, mag, k, 2.0, eights)


@pytest.mark.parametrize("c,n,k", [([3, 5, 2], 72, 264), ([60, 33, 45], 520, 1800), ([301, 77, 200], 264, 40),
                                   ([3001, 2500, 1], 2056, 1032)])
def test_not_finite_stays_in_its_row_and_group(c, n, k):
    """An infinity and a NaN in the last row of the first group: no other row
    and no other group's weight gradient sees them."""
    g = gen_of(n + k)
    rows, off, last = sum(c), offsets_of(c), c[0] - 1
    x, w, dy = randn(g, rows, k), randn(g, len(c), n, k), randn(g, rows, n)
    x[last, 0], dy[last, 1] = float("nan"), float("inf")
    others = torch.arange(rows, device="cuda") != last
    got = B.situ_moe_grouped_matmul(x, w, off)
    want, mag = grouped_ref(x, w, c)
    assert torch.isnan(got[last]).all()
    close(got[others], want[others], mag[others], k)
    got = B.situ_moe_grouped_matmul_dgrad(dy, w, off)
    want, mag = grouped_ref(dy, w.transpose(1, 2), c)
    assert not torch.isfinite(got[last]).any()
    close(got[others], want[others], mag[others], n)
    dw = B.situ_moe_grouped_matmul_wgrad(dy, x, off)
    assert torch.isnan(dw[0, :, 0]).all() and not torch.isfinite(dw[0, 1]).any()
    lo = c[0]
    for e, m in enumerate(c[1:], 1):
        xe, de = x[lo:lo + m].to(D), dy[lo:lo + m].to(D)
        close(dw[e], de.t() @ xe, de.abs().t() @ xe.abs(), m)
        lo += m
    k8 = k // 16 * 16
    a, sa, w8, sw = fp8_inputs(g, rows, len(c), n, k8)
    want, mag, eights = fp8_ref(a, sa, w8, sw, c)
    a[last, 3] = 0x7f
    for out in (BF, F32):
        got = B.situ_moe_matmul_fp8_block128(a, sa, w8, sw, offsets=off, out_dtype=out)
        assert torch.isnan(got[last]).all()
        close(got[others], want[others], mag[others], k8, 2.0, eights[others])


@pytest.mark.parametrize("c,n,k", [([900, 1, 0, 1300], 2056, 2056), ([700, 90, 333], 264, 1032), ([5000], 32, 520),
                                   ([40, 0, 100, 64, 65], 136, 1544)])
@pytest.mark.parametrize("gather", [False, True])
def test_wgrad_tile_shapes(c, n, k, gather):
    g = gen_of(n + k)
    rows, off = sum(c), offsets_of(c)
    dy = randn(g, rows, n)
    pairs, x_div = None, 0
    x = xs = randn(g, rows, k)
    if gather:
        pairs = torch.randperm(2 * rows, generator=g, device="cuda")[:rows].to(torch.int32)
        x_div, xs = 4, randn(g, -(-2 * rows // 4), k)
        x = xs[pairs.long() // 4]
    dw = B.situ_moe_grouped_matmul_wgrad(dy, xs, off, pairs=pairs, x_div=x_div)
    lo = 0
    for e, m in enumerate(c):
        xe, de = x[lo:lo + m].to(D), dy[lo:lo + m].to(D)
        close(dw[e], de.t() @ xe, de.abs().t() @ xe.abs(), m)
        lo += m


def test_pairs_at_size():
    """Gathered and scattered rows through the large tiles, more experts than rows, the most experts."""
    c, n, k = [2100, 0, 1, 1995], 2056, 1032
    g = gen_of(21)
    rows, top_k = sum(c), 4
    tokens = -(-rows * 2 // top_k)
    pairs = torch.randperm(tokens * top_k, generator=g, device="cuda")[:rows].to(torch.int32)
    xt, w = randn(g, tokens, k), randn(g, len(c), n, k)
    got = torch.full((tokens * top_k, n), 3.0, dtype=BF, device="cuda")
    B.situ_moe_grouped_matmul(xt, w, offsets_of(c), pairs=pairs, x_div=top_k, out_div=1, out=got)
    want, mag = grouped_ref(xt[pairs.long() // top_k], w, c)
    close(got[pairs.long()], want, mag, k)
    rest = torch.ones(tokens * top_k, dtype=torch.bool, device="cuda")
    rest[pairs.long()] = False
    assert (got[rest] == 3.0).all()
    c = [(i * 7919) % 3 // 2 for i in range(1024)]
    x, w, dy = randn(g, sum(c), 72), randn(g, 1024, 24, 72), randn(g, sum(c), 24)
    want, mag = grouped_ref(x, w, c)
    close(B.situ_moe_grouped_matmul(x, w, offsets_of(c)), want, mag, 72)
    want, mag = grouped_ref(dy, w.transpose(1, 2), c)
    close(B.situ_moe_grouped_matmul_dgrad(dy, w, offsets_of(c)), want, mag, 24)
    dw = B.situ_moe_grouped_matmul_wgrad(dy, x, offsets_of(c))
    expert = torch.repeat_interleave(torch.arange(1024, device="cuda"), torch.tensor(c, device="cuda"))
    want = torch.zeros(1024, 24, 72, dtype=D, device="cuda")
    want[expert] = dy.to(D)[:, :, None] * x.to(D)[:, None, :]
    assert torch.equal(dw.to(D), want)              # one row each: exact


def test_no_rows():
    g = gen_of(4)
    w = randn(g, 3, 16, 32)
    off = torch.zeros(4, dtype=torch.int32, device="cuda")
    empty = torch.empty(0, 32, dtype=BF, device="cuda")
    assert B.situ_moe_grouped_matmul(empty, w, off).shape == (0, 16)
    assert B.situ_moe_grouped_matmul_dgrad(torch.empty(0, 16, dtype=BF, device="cuda"), w, off).shape == (0, 32)
    dw = torch.full((3, 16, 32), 7.0, device="cuda")
    B.situ_moe_grouped_matmul_wgrad(torch.empty(0, 16, dtype=BF, device="cuda"), empty, off, out=dw)
    assert (dw == 0).all()
    # rows, but all of them outside the groups
    x = randn(g, 5, 32)
    out = torch.full((5, 16), 3.0, dtype=BF, device="cuda")
    B.situ_moe_grouped_matmul(x, w, off, out=out)
    assert (out == 3.0).all()
    c, s = B.situ_moe_quantize_fp8_block128(torch.empty(0, 128, dtype=BF, device="cuda"))
    assert c.shape == (0, 128) and s.shape == (0, 1)


def test_wrong_offsets_and_pairs_stay_inside():
    """Offsets that do not ascend and pairs outside the arrays: unspecified rows, no access outside, rows of no
    valid index untouched."""
    g = gen_of(6)
    x, w, dy = randn(g, 100, 64), randn(g, 4, 128, 64), randn(g, 100, 128)
    for off in ([0, 50, 20, 100, 100], [-5, 10, 1000, 2 ** 31 - 1, 100], [100, 100, 0, 0, 0]):
        o = torch.tensor(off, dtype=torch.int32, device="cuda")
        B.situ_moe_grouped_matmul(x, w, o)
        B.situ_moe_grouped_matmul_dgrad(dy, w, o)
        B.situ_moe_grouped_matmul_wgrad(dy, x, o)
    torch.cuda.synchronize()
    pairs = torch.arange(100, dtype=torch.int32, device="cuda")
    pairs[7], pairs[8], pairs[9] = -1, 2 ** 31 - 1, 100
    out = torch.full((100, 128), 3.0, dtype=F32, device="cuda")
    off = offsets_of([10, 20, 30, 40])
    B.situ_moe_grouped_matmul(x, w, off, pairs=pairs, x_div=1, out_div=1, out=out)
    want, mag = grouped_ref(x, w, [10, 20, 30, 40])
    ok = torch.ones(100, dtype=torch.bool, device="cuda")
    ok[7:10] = False
    close(out[ok], want[ok], mag[ok], 64)
    assert (out[7:10] == 3.0).all()
    B.situ_moe_grouped_matmul_wgrad(dy, x, off, pairs=pairs, x_div=1, dy_div=1)
    torch.cuda.synchronize()


def test_arrays_beyond_4_gib():
    rows_x, k, n = 720_000, 3584, 16                # 5.2 GB of x
    g = gen_of(8)
    x = torch.zeros(rows_x, k, dtype=BF, device="cuda")
    take = torch.tensor([0, rows_x - 1, 599_186, 650_001, 3, rows_x - 2], dtype=torch.int32, device="cuda")
    x[take.long()] = randn(g, 6, k)
    w = randn(g, 2, n, k)
    c = [4, 2]
    got = B.situ_moe_grouped_matmul(x, w, offsets_of(c), pairs=take, x_div=1, out_dtype=F32)
    want, mag = grouped_ref(x[take.long()], w, c)
    close(got, want, mag, k)
    dy = randn(g, 6, n)
    dw = B.situ_moe_grouped_matmul_wgrad(dy, x, offsets_of(c), pairs=take, x_div=1)
    close(dw[0], dy[:4].to(D).t() @ x[take[:4].long()].to(D), dy[:4].to(D).abs().t() @ x[take[:4].long()].to(D).abs(), 4)
    dx = x                                          # written rows beyond 4 GiB
    B.situ_moe_grouped_matmul_dgrad(dy, w, offsets_of(c), pairs=take, out_div=1, out=dx)
    want, mag = grouped_ref(dy, w.transpose(1, 2), c)
    close(dx[take.long()], want, mag, n)
    assert (dx[1] == 0).all() and (dx[rows_x - 3] == 0).all()


def test_gathered_rows_beyond_2_gib():
    """Offsets with the highest of 32 bits set, through the large tiles."""
    rows_x, k, n = 500_000, 4096, 2056              # 4.1 GB of x
    c = [2500, 1500]
    g = gen_of(22)
    x = torch.zeros(rows_x, k, dtype=BF, device="cuda")
    take = (torch.randperm(rows_x // 2, generator=g, device="cuda")[:4000] * 2 + 1).to(torch.int32)   # the last row's parity
    take[5] = rows_x - 1
    x[take.long()] = randn(g, 4000, k)
    w, dy = randn(g, 2, n, k), randn(g, 4000, n)
    want, mag = grouped_ref(x[take.long()], w, c)
    close(B.situ_moe_grouped_matmul(x, w, offsets_of(c), pairs=take, x_div=1), want, mag, k)
    dw = B.situ_moe_grouped_matmul_wgrad(dy, x, offsets_of(c), pairs=take, x_div=1)
    xe, de = x[take[:2500].long()].to(D), dy[:2500].to(D)
    close(dw[0], de.t() @ xe, de.abs().t() @ xe.abs(), 2500)


# ---------------------------------------------------------------- refusals

def refused(status, f):
    with pytest.raises(B.SituMoeError) as e:
        f()
    assert e.value.status_name == status, e.value


def test_refusals():
    x = torch.zeros(10, 64, dtype=BF, device="cuda")
    w = torch.zeros(3, 32, 64, dtype=BF, device="cuda")
    dy = torch.zeros(10, 32, dtype=BF, device="cuda")
    off = torch.zeros(4, dtype=torch.int32, device="cuda")
    pairs = torch.zeros(10, dtype=torch.int32, device="cuda")
    f, d, g = B.situ_moe_grouped_matmul, B.situ_moe_grouped_matmul_dgrad, B.situ_moe_grouped_matmul_wgrad
    for bad in ("SITU_E_NULL_ARG", None), ("SITU_E_DEVICE", x.cpu()), ("SITU_E_BAD_SHAPE", x.float()), \
               ("SITU_E_BAD_SHAPE", x[0]), ("SITU_E_BAD_SHAPE", x.t().contiguous().t()), ("SITU_E_BAD_SHAPE", x[:, :56]):
        refused(bad[0], lambda: f(bad[1], w, off))
    refused("SITU_E_BAD_SHAPE", lambda: f(x, w, off.long()))
    refused("SITU_E_BAD_SHAPE", lambda: f(x, w, off[:3]))
    refused("SITU_E_NULL_ARG", lambda: f(x, w))
    refused("SITU_E_NULL_ARG", lambda: f(x, w, off, x_div=2))
    refused("SITU_E_NULL_ARG", lambda: f(x, w, off, pairs=pairs, out_div=1))       # needs out
    refused("SITU_E_BAD_SHAPE", lambda: f(x, w, off, pairs=pairs, out_div=2, out=dy))
    refused("SITU_E_BAD_SHAPE", lambda: f(x, w, off, pairs=pairs, x_div=-1))
    refused("SITU_E_BAD_SHAPE", lambda: f(x, w.transpose(1, 2), off))
    refused("SITU_E_BAD_SHAPE", lambda: f(x, w, off, pairs=pairs[:5]))            # 5 positions, 10 rows
    refused("SITU_E_BAD_SHAPE", lambda: f(x, w, off, out=dy[:5]))
    refused("SITU_E_BAD_SHAPE", lambda: f(x, w, off, out=dy, out_dtype=F32))
    refused("SITU_E_UNSUPPORTED", lambda: f(x, w, off, out_dtype=torch.float16))
    refused("SITU_E_BAD_SHAPE", lambda: f(x[:, :60].contiguous(), w[:, :, :60].contiguous(), off))
    refused("SITU_E_BAD_SHAPE", lambda: f(x.view(-1)[4:4 + 9 * 64].view(9, 64), w, off))   # rows off 16 bytes
    refused("SITU_E_BAD_SHAPE", lambda: f(x[:1].expand(10, 64), w, off))
    refused("SITU_E_BAD_SHAPE", lambda: d(dy[:, :28], w[:, :28].contiguous(), off))
    refused("SITU_E_BAD_SHAPE", lambda: d(x, w, off))
    refused("SITU_E_BAD_SHAPE", lambda: g(dy[:9], x, off))
    refused("SITU_E_BAD_SHAPE", lambda: g(dy, x, off, out=torch.zeros(3, 32, 56, device="cuda")))
    refused("SITU_E_BAD_SHAPE", lambda: B.situ_moe_quantize_fp8_block128(x[:, :40]))
    refused("SITU_E_BAD_SHAPE", lambda: B.situ_moe_quantize_fp8_block128(x.half()))
    a, s = B.situ_moe_quantize_fp8_block128(x)
    w8, ws = torch.zeros(32, 64, dtype=torch.uint8, device="cuda"), torch.ones(1, 1, device="cuda")
    m = B.situ_moe_matmul_fp8_block128
    assert m(a.view(F8), s, w8.view(F8), ws).shape == (10, 32)
    refused("SITU_E_BAD_SHAPE", lambda: m(a, s[:5], w8, ws))
    refused("SITU_E_BAD_SHAPE", lambda: m(a, s, w8, ws.double()))
    refused("SITU_E_BAD_SHAPE", lambda: m(a, s, w8, ws, offsets=off))
    refused("SITU_E_BAD_SHAPE", lambda: m(a, s, w8[None], ws[None]))
    refused("SITU_E_BAD_SHAPE", lambda: m(a[:, :40], s, w8[:, :40].contiguous(), ws))
    refused("SITU_E_NULL_ARG", lambda: m(a, None, w8, ws))
    refused("SITU_E_UNSUPPORTED", lambda: m(a, s, w8, ws, out_dtype=torch.float16))


def test_refusal_of_a_scalar():
    s = torch.zeros((), dtype=BF, device="cuda")
    w = torch.zeros(1, 32, 64, dtype=BF, device="cuda")
    refused("SITU_E_BAD_SHAPE", lambda: B.situ_moe_grouped_matmul(s, w))
    refused("SITU_E_BAD_SHAPE", lambda: B.situ_moe_grouped_matmul_dgrad(s, w))
    refused("SITU_E_BAD_SHAPE", lambda: B.situ_moe_grouped_matmul_wgrad(s, s))
    refused("SITU_E_BAD_SHAPE", lambda: B.situ_moe_quantize_fp8_block128(s))


def test_refusal_of_offsets_without_groups():
    x, dy = torch.zeros(10, 64, dtype=BF, device="cuda"), torch.zeros(10, 32, dtype=BF, device="cuda")
    off = torch.zeros(4, dtype=torch.int32, device="cuda")
    for n in (0, 1):
        refused("SITU_E_BAD_SHAPE", lambda: B.situ_moe_grouped_matmul_wgrad(dy, x, off[:n]))


# ------------------------------------------------------------ streams, graphs

def test_deterministic_and_other_stream():
    g = gen_of(9)
    c = COUNTS["ragged"]
    x, w, dy = randn(g, sum(c), 328), randn(g, len(c), 200, 328), randn(g, sum(c), 200)
    off = offsets_of(c)
    first = (B.situ_moe_grouped_matmul(x, w, off), B.situ_moe_grouped_matmul_dgrad(dy, w, off),
             B.situ_moe_grouped_matmul_wgrad(dy, x, off))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    again = (B.situ_moe_grouped_matmul(x, w, off, stream=s), B.situ_moe_grouped_matmul_dgrad(dy, w, off, stream=s),
             B.situ_moe_grouped_matmul_wgrad(dy, x, off, stream=s.cuda_stream))
    s.synchronize()
    for a, b in zip(first, again):
        assert torch.equal(a, b)


def test_two_calls_at_once():
    """The kernels hold no state: calls on two streams give what they give alone."""
    g = gen_of(31)
    c = [1000, 300, 0, 748]
    x, w = randn(g, 2048, 520), randn(g, 4, 776, 520)
    y, v = randn(g, 2048, 520), randn(g, 4, 776, 520)
    off = offsets_of(c)
    alone = B.situ_moe_grouped_matmul(x, w, off), B.situ_moe_grouped_matmul(y, v, off)
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    got = []
    for _ in range(4):
        got.append((B.situ_moe_grouped_matmul(x, w, off, stream=s), B.situ_moe_grouped_matmul(y, v, off, stream=t)))
    torch.cuda.synchronize()
    for p in got:
        assert torch.equal(p[0], alone[0]) and torch.equal(p[1], alone[1])


def test_graph_replay():
    """Both directions and the FP8 chain captured once; replayed on new inputs and other group sizes."""
    g = gen_of(10)
    c = [30, 0, 100, 70]
    x, w, dy = randn(g, 200, 256), randn(g, 4, 136, 256), randn(g, 200, 136)
    w8, sw = B.situ_moe_quantize_fp8_block128(w.view(-1, 256))
    w8, sw = w8.view(4, 136, 256), torch.rand(4, 2, 2, device="cuda")
    off = offsets_of(c)

    def chain():
        a, sa = B.situ_moe_quantize_fp8_block128(x)
        return (B.situ_moe_grouped_matmul(x, w, off), B.situ_moe_grouped_matmul_dgrad(dy, w, off),
                B.situ_moe_grouped_matmul_wgrad(dy, x, off), B.situ_moe_matmul_fp8_block128(a, sa, w8, sw, offsets=off))

    chain()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = chain()
    for i, c in enumerate(([30, 0, 100, 70], [0, 200, 0, 0], [1, 99, 99, 1])):
        x.copy_(randn(g, 200, 256))
        dy.copy_(randn(g, 200, 136))
        off.copy_(offsets_of(c))
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(held, chain()):
            assert torch.equal(a, b), i


# ------------------------------------------------- the set as it is used together

def test_adapter_beside_the_layer():
    """A LoRA adapter on gate_up: its two products over the layer's own routing tables make gate_up_lora_delta; the
    down adapter's first product reads activation_lora_input.  The layer's output equals the one it gives for the same
    delta made by torch."""
    spec = S.spec_of(dict(S.CONFIGS[1], T=24, seed=77))
    inp = S.generate(spec)
    from gpu_helpers import dev
    T, H, I, k, E = spec["T"], spec["H"], spec["I"], spec["k"], spec["E_l"]
    r = 16
    g = gen_of(11)
    A = (randn(g, E, r, H).float() / H ** 0.5).to(BF)
    Bm = (randn(g, E, 2 * I, r).float() * 0.25).to(BF)
    prob = B.make_problem(num_tokens=T, hidden_size=H, intermediate_size=I, num_experts=spec["E_g"],
                          local_expert_offset=spec["off"], local_num_experts=E, top_k=k)
    plan = B.situ_moe_plan(prob)
    ws = B.new_workspace(plan)
    d = {key: dev(inp[key]) for key in ("hidden_states", "topk_ids", "topk_weights", "w1", "w1_scale", "w2",
                                        "w2_scale", "situ_beta", "situ_linear_beta", "alpha_gate", "alpha_up")}
    d["topk_ids"] = d["topk_ids"].to(torch.int32)
    out = torch.empty((T, H), device="cuda")
    delta = torch.zeros((T * k, 2 * I), dtype=BF, device="cuda")
    h = torch.empty((T * k, I), dtype=BF, device="cuda")
    ts = B.make_tensors(prob, out=out, gate_up_lora_delta=delta, activation_lora_input=h, **d)
    B.situ_moe_route(plan, ts, ws)
    off = B.workspace_view(plan, ws, "offsets", torch.int32, (E + 1,)).clone()
    perm = B.workspace_view(plan, ws, "perm", torch.int32, (T * k,)).clone()
    t = B.situ_moe_grouped_matmul(d["hidden_states"], A, off, pairs=perm, x_div=k)
    B.situ_moe_grouped_matmul(t, Bm, off, pairs=perm, out_div=1, out=delta)
    B.situ_moe_run(plan, ts, ws)
    torch.cuda.synchronize()
    local = int(off[-1])
    expert = torch.repeat_interleave(torch.arange(E, device="cuda"), off.diff().long(), output_size=local)
    p = perm[:local].long()
    want = torch.zeros_like(delta)
    x64 = d["hidden_states"].to(D)[p // k]
    t64 = (x64[:, None, :] @ A.to(D)[expert].transpose(1, 2)).squeeze(1)
    mag = (x64.abs()[:, None, :] @ A.to(D).abs()[expert].transpose(1, 2)).squeeze(1)
    close(t[:local], t64, mag, H)
    tb = t[:local].to(D)
    d64 = (tb[:, None, :] @ Bm.to(D)[expert].transpose(1, 2)).squeeze(1)
    mag = (tb.abs()[:, None, :] @ Bm.to(D).abs()[expert].transpose(1, 2)).squeeze(1)
    close(delta[p], d64, mag, r)
    rest = torch.ones(T * k, dtype=torch.bool, device="cuda")
    rest[p] = False
    assert (delta[rest] == 0).all()
    # the layer reads the delta as it would any other
    want[p] = delta[p]
    out2 = torch.empty_like(out)
    ts2 = B.make_tensors(prob, out=out2, gate_up_lora_delta=want, activation_lora_input=h, **d)
    B.situ_moe_run(plan, ts2, ws)
    torch.cuda.synchronize()
    assert torch.equal(out, out2) and torch.isfinite(out).all()
    # the down adapter's first product on the rows the layer handed back
    A2 = (randn(g, E, r, I).float() / I ** 0.5).to(BF)
    t2 = B.situ_moe_grouped_matmul(h, A2, off, pairs=perm, x_div=1)
    h64 = h.to(D)[p]
    close(t2[:local], (h64[:, None, :] @ A2.to(D)[expert].transpose(1, 2)).squeeze(1),
          (h64.abs()[:, None, :] @ A2.to(D).abs()[expert].transpose(1, 2)).squeeze(1), I)


def test_fp8_experts_chain():
    """An expert layer of FP8 weights: quantize, gate and up, SwiGLU, quantize, down."""
    c = [9, 0, 40, 3]
    H, I = 512, 192
    g = gen_of(12)
    rows = sum(c)
    off = offsets_of(c)
    x = randn(g, rows, H)
    _, _, w1, s1 = fp8_inputs(g, 1, 4, 2 * I, H)
    _, _, w2, s2 = fp8_inputs(g, 1, 4, H, I)
    s1, s2 = s1 * 1e-3, s2 * 1e-3
    a, sa = B.situ_moe_quantize_fp8_block128(x)
    gu = B.situ_moe_matmul_fp8_block128(a, sa, w1, s1, offsets=off, out_dtype=F32)
    want, mag, eights = fp8_ref(a, sa, w1, s1, c)
    close(gu, want, mag, H, 2.0, eights)
    h = (torch.nn.functional.silu(gu[:, :I]) * gu[:, I:]).to(BF)
    b, sb = B.situ_moe_quantize_fp8_block128(h)
    y = B.situ_moe_matmul_fp8_block128(b, sb, w2, s2, offsets=off)
    want, mag, eights = fp8_ref(b, sb, w2, s2, c)
    close(y, want, mag, I, 2.0, eights)
