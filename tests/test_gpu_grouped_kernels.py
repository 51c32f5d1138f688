"""Every kernel of the products beside the layer on calls that are known to
reach it (tests/grouped_kernels.py), against the formulas in 64 bits.

Tolerances are those derived in test_gpu_grouped.  Rows of no group hold NaN
or infinities, as do rows that no position looks up, and pairs of positions of
no group are no rows; groups hold no row, one, and rows that end inside steps
and tiles.  A repeated call gives the same bits.
"""

import pytest
import torch

import block_scaled_mxfp4_amd as B
from grouped_kernels import CASES, case_id, kernel_of, rows_of
from test_gpu_grouped import BF, D, F32, close, fp8_inputs, fp8_ref, gen_of, grouped_ref, offsets_of, randn

pytestmark = pytest.mark.gpu


def takes(kernel, *args, **kw):
    cus = torch.cuda.get_device_properties(0).multi_processor_count
    assert kernel_of(*args, cus=cus, **kw) == kernel


def layout(counts):
    """Rows, groups, rows in groups, rows per group, offsets."""
    rows, experts = rows_of(counts)
    per = [counts] if isinstance(counts, int) else counts
    return rows, experts, sum(per), per, None if isinstance(counts, int) else offsets_of(per)


def same(call):
    first = call()
    again = call()
    assert torch.equal(first, again)
    return first


@pytest.mark.parametrize("case", [c for c in CASES if c[0] in ("fwd", "dgrad")], ids=case_id)
def test_product_and_dgrad(case):
    op, _, kernel, counts, n, k, _ = case
    rows, experts, held, per, off = layout(counts)
    g = gen_of(n + 3 * k)
    fwd = op == "fwd"
    depth, cols = (k, n) if fwd else (n, k)
    t, w = randn(g, rows, depth, pad=8), randn(g, experts, n, k)
    t[held:] = float("nan") if fwd else float("inf")
    for e, c in enumerate(per):
        if c == 0:
            w[e] = float("nan")
    want, mag = grouped_ref(t[:held], w if fwd else w.transpose(1, 2), per)
    for out in (BF, F32):
        takes(kernel, op, rows, experts, n, k, f32=out == F32, offsets=off is not None)
        call = B.situ_moe_grouped_matmul if fwd else B.situ_moe_grouped_matmul_dgrad
        got = torch.full((rows, cols + 5), 3.0, dtype=out, device="cuda")
        call(t, w, off, out=got[:, :cols])
        first = got.clone()
        got[:held, :cols] = 0
        call(t, w, off, out=got[:, :cols])
        assert torch.equal(first, got)
        close(got[:held, :cols], want, mag, depth)
        assert (got[held:] == 3.0).all() and (got[:, cols:] == 3.0).all()
        dense = same(lambda: call(t, w, off, out_dtype=out)[:held])      # rows on 16 bytes where cols allows
        assert torch.equal(dense, got[:held, :cols])


@pytest.mark.parametrize("case", [c for c in CASES if c[0] == "fp8"], ids=case_id)
def test_fp8(case):
    _, f32, kernel, counts, n, k, _ = case
    rows, experts, held, per, off = layout(counts)
    out = F32 if f32 else BF
    takes(kernel, "fp8", rows, experts, n, k, f32=f32, offsets=off is not None)
    a, sa, w, sw = fp8_inputs(gen_of(n + 5 * k), rows, experts, n, k, 16)
    a[held:] = 0x7f
    for e, c in enumerate(per):
        if c == 0:
            w[e] = 0x7f
    if off is None:
        got = same(lambda: B.situ_moe_matmul_fp8_block128(a, sa, w[0], sw[0], out_dtype=out))
    else:
        got = torch.full((rows, n + 3), 3.0, dtype=out, device="cuda")
        same(lambda: B.situ_moe_matmul_fp8_block128(a, sa, w, sw, offsets=off, out=got[:, :n]).clone())
        assert (got[held:] == 3.0).all() and (got[:, n:] == 3.0).all()
        got = got[:, :n]
    want, mag, eights = fp8_ref(a[:held], sa, w, sw, per)
    few = "few" in kernel
    close(got[:held], want, mag, k, 2.0, None if few or f32 else eights)


def wgrad_inputs(g, rows, held, n, k, sides):
    """dy and x as the call takes them and row by row, and its arguments."""
    dy, x = randn(g, rows, n, pad=8), randn(g, rows, k, pad=16)
    dy[held:], x[held:] = float("inf"), float("nan")
    if not sides:
        return dy, x, dy, x, {}
    order = torch.randperm(2 * rows, generator=g, device="cuda")[:rows].to(torch.int32)
    pairs = order.clone()
    pairs[held:] = torch.tensor([-1, 2 ** 31 - 1, 2 * rows], dtype=torch.int32, device="cuda")[:rows - held]
    kw = dict(pairs=pairs)
    dys, xs = dy, x
    if "y" in sides:
        dys = torch.full((2 * rows, n), float("inf"), dtype=BF, device="cuda")
        dys[order[:held].long()] = dy[:held]
        kw["dy_div"] = 1
    if "x" in sides:
        xs = randn(g, -(-2 * rows // 4), k)
        x = xs[order.long() // 4]
        kw["x_div"] = 4
    return dys, xs, dy, x, kw


def check_dw(dw, dy, x, per):
    lo = 0
    for e, m in enumerate(per):
        xe, de = x[lo:lo + m].to(D), dy[lo:lo + m].to(D)
        close(dw[e], de.t() @ xe, de.abs().t() @ xe.abs(), m)
        lo += m


@pytest.mark.parametrize("case", [c for c in CASES if c[0] == "wgrad"], ids=case_id)
def test_wgrad(case):
    _, _, kernel, counts, n, k, sides = case
    rows, experts, held, per, off = layout(counts)
    dys, xs, dy, x, kw = wgrad_inputs(gen_of(n + 7 * k), rows, held, n, k, sides)
    for out in (F32, BF):
        takes(kernel, "wgrad", rows, experts, n, k, f32=out == F32, offsets=off is not None, sides=sides,
              x_rows=xs.shape[0])
        check_dw(same(lambda: B.situ_moe_grouped_matmul_wgrad(dys, xs, off, out_dtype=out, **kw)), dy, x, per)


def test_wgrad_of_rows_beyond_2_gib():
    """Looked-up rows whose 32-bit byte offsets have the highest bit set, through the 256 x 256 tiles."""
    rows_x, n, k, c = 500_000, 4104, 4096, [2500, 0, 1500]         # 4.1 GB of x
    takes("grouped_pair_kernel indexed", "wgrad", 4000, 3, n, k, f32=True, sides="x", x_rows=rows_x)
    g = gen_of(23)
    x = torch.zeros(rows_x, k, dtype=BF, device="cuda")
    take = (rows_x - 1 - torch.randperm(200_000, generator=g, device="cuda")[:4000]).to(torch.int32)   # past 2^31
    take[7] = 0
    x[take.long()] = randn(g, 4000, k)
    dy = randn(g, 4000, n)
    check_dw(B.situ_moe_grouped_matmul_wgrad(dy, x, offsets_of(c), pairs=take, x_div=1), dy, x[take.long()], c)


@pytest.mark.parametrize("sides", ["", "x"])
def test_wgrad_replayed_with_other_groups(sides):
    """The 256 x 256 weight gradient captured once and replayed on other groups, rows and lookups."""
    n, k, rows, experts = 2568, 2312, 2040, 6
    at = " indexed" if sides else ""
    takes("grouped_pair_kernel" + at, "wgrad", rows, experts, n, k, f32=True, sides=sides, x_rows=rows // 2)
    splits = [[0, 700, 130, 1, 0, 1200], [2040, 0, 0, 0, 0, 0], [64, 128, 192, 65, 129, 1000], [0] * 6]
    g = gen_of(29)
    off = offsets_of(splits[0])
    dys, xs, dy, x, kw = wgrad_inputs(g, rows, rows, n, k, sides)
    call = lambda: B.situ_moe_grouped_matmul_wgrad(dys, xs, off, **kw)   # noqa: E731
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = call()
    for i, per in enumerate(splits):
        dys, xs, dy, x, new = [t.copy_(u) if torch.is_tensor(t) else u for t, u in
                               zip((dys, xs, dy.clone(), x.clone(), kw), wgrad_inputs(g, rows, rows, n, k, sides))]
        if sides:
            kw["pairs"].copy_(new["pairs"])
        off.copy_(offsets_of(per))
        graph.replay()
        torch.cuda.synchronize()
        check_dw(held, dy, x, per)
        assert torch.equal(held, call()), i
