"""What the FP8 and grouped products refuse, on the host (no GPU needed, no
kernel is launched)."""

import ctypes
import os
import subprocess

import pytest
import torch

import block_scaled_mxfp4_amd as B

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "situ_moe.h")
FAKE = 1 << 20          # never dereferenced: every case fails on the host first


def test_struct_layout_matches_header(tmp_path):
    py = {"situ_moe_fp8_matmul_t": B.SituMoeFp8Matmul, "situ_moe_grouped_t": B.SituMoeGrouped}
    lines = ['#include <stdio.h>', '#include <stddef.h>', f'#include "{HEADER}"', "int main(void) {"]
    for st, cls in py.items():
        lines.append(f'printf("{st} size %zu\\n", sizeof({st}));')
        lines += [f'printf("{st} {f} %zu\\n", offsetof({st}, {f}));' for f, _ in cls._fields_]
    c = tmp_path / "layout.c"
    c.write_text("\n".join(lines + ["return 0; }"]))
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", str(c), "-o", str(exe)], check=True)
    out = subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split("\n")
    n = 0
    for line in filter(None, out):
        st, f, v = line.split()
        assert (ctypes.sizeof(py[st]) if f == "size" else getattr(py[st], f).offset) == int(v), (st, f)
        n += 1
    assert n == sum(len(c._fields_) + 1 for c in py.values())



def _quantize(x=FAKE, rows=4, cols=256, stride=256, codes=FAKE, scales=FAKE):
    return B.load().situ_moe_quantize_fp8_block128(x, rows, cols, stride, codes, scales, None)


@pytest.mark.parametrize("kw,want", [
    (dict(rows=-1), 2), (dict(cols=0), 2), (dict(cols=40), 2), (dict(stride=255), 2), (dict(stride=260), 2),
    (dict(x=FAKE + 8), 2), (dict(codes=FAKE + 4), 2), (dict(scales=FAKE + 2), 2), (dict(x=None), 1),
    (dict(codes=None), 1), (dict(scales=None), 1), (dict(rows=(1 << 24) + 1), 3), (dict(cols=(1 << 18) + 16), 3),
    (dict(rows=0, x=None), 0), (dict(stride=1 << 41), 2)])
def test_quantize_refusals(kw, want):
    assert _quantize(**kw) == want, B.situ_moe_last_error()


def _fp8(**kw):
    base = dict(rows=4, n=200, k=256, experts=1, out_dtype=B.OUT_BF16, a_stride=256, a_scale_stride=2, out_stride=200,
                a=FAKE, a_scale=FAKE, w=FAKE, w_scale=FAKE, out=FAKE)
    return B.load().situ_moe_matmul_fp8_block128(ctypes.byref(B.SituMoeFp8Matmul(**dict(base, **kw))), None)


@pytest.mark.parametrize("kw,want", [
    (dict(rows=-1), 2), (dict(n=0), 2), (dict(k=0), 2), (dict(k=24), 2), (dict(experts=0), 2), (dict(out_dtype=2), 3),
    (dict(reserved=1), 2), (dict(experts=2), 1), (dict(experts=1025, offsets=FAKE), 3), (dict(n=(1 << 18) + 1), 3),
    (dict(rows=(1 << 24) + 1), 3), (dict(a=None), 1), (dict(a_scale=None), 1), (dict(w=None), 1),
    (dict(w_scale=None), 1), (dict(out=None), 1), (dict(a=FAKE + 8), 2), (dict(w=FAKE + 4), 2), (dict(out=FAKE + 1), 2),
    (dict(a_scale=FAKE + 2), 2), (dict(w_scale=FAKE + 1), 2), (dict(offsets=FAKE + 2), 2), (dict(a_stride=240), 2),
    (dict(a_stride=264), 2), (dict(a_scale_stride=1), 2), (dict(out_stride=199), 2), (dict(rows=0, a=None), 0),
    (dict(a_scale_stride=1 << 22), 3), (dict(a_scale_stride=1 << 32), 3), (dict(a_scale_stride=1 << 41), 2)])
def test_fp8_matmul_refusals(kw, want):
    assert _fp8(**kw) == want, B.situ_moe_last_error()
    assert B.load().situ_moe_matmul_fp8_block128(None, None) == 1


def _grouped(fn, **kw):
    base = dict(rows=4, n=64, k=128, experts=3, x_rows=4, y_rows=4, out_dtype=B.OUT_BF16, x_stride=128, y_stride=64,
                offsets=FAKE, x=FAKE, y=FAKE, w=FAKE)
    return getattr(B.load(), "situ_moe_grouped_matmul" + fn)(ctypes.byref(B.SituMoeGrouped(**dict(base, **kw))), None)


@pytest.mark.parametrize("fn", ["", "_dgrad", "_wgrad"])
@pytest.mark.parametrize("kw,want", [
    (dict(rows=-1), 2), (dict(n=0), 2), (dict(k=0), 2), (dict(k=12, x_stride=16), 2), (dict(experts=0), 2),
    (dict(experts=1025), 3), (dict(offsets=None), 1), (dict(offsets=FAKE + 1), 2), (dict(out_dtype=7), 3),
    (dict(reserved=3), 2), (dict(x=None), 1), (dict(y=None), 1), (dict(w=None), 1), (dict(x=FAKE + 1), 2),
    (dict(y=FAKE + 1), 2), (dict(w=FAKE + 1), 2), (dict(x_stride=120), 2), (dict(y_stride=56), 2), (dict(x_div=-1), 2),
    (dict(y_div=-1), 2), (dict(x_div=1), 1), (dict(y_div=1), 1), (dict(x_div=1, pairs=FAKE + 2), 2),
    (dict(x_div=1, pairs=FAKE, x_rows=0), 2), (dict(y_div=1, pairs=FAKE, y_rows=0), 2),
    (dict(rows=(1 << 24) + 1), 3), (dict(n=1 << 19, y_stride=1 << 19), 3), (dict(k=1 << 19, x_stride=1 << 19), 3)])
def test_grouped_refusals(fn, kw, want):
    assert _grouped(fn, **kw) == want, B.situ_moe_last_error()
    assert getattr(B.load(), "situ_moe_grouped_matmul" + fn)(None, None) == 1


def test_grouped_refusals_of_one_direction():
    assert _grouped("", y_div=2, pairs=FAKE) == 2                 # a written row for two positions
    assert _grouped("_dgrad", x_div=2, pairs=FAKE) == 2
    assert _grouped("_dgrad", n=60, y_stride=64) == 2             # n a multiple of 8 where dy is read along it
    assert _grouped("_wgrad", n=60, y_stride=64) == 2
    assert _grouped("", x=FAKE + 8) == 2 and _grouped("_dgrad", y=FAKE + 8) == 2 and _grouped("_wgrad", y=FAKE + 8) == 2
    assert _grouped("", x_stride=132) == 2 and _grouped("_wgrad", y_stride=68) == 2
    assert _grouped("", rows=0, x=None, y=None, w=None) == 0
    assert _grouped("_dgrad", rows=0, x=None, y=None, w=None) == 0
    assert _grouped("_wgrad", rows=0, x=None, y=None, w=None) == 1   # dw of no rows is written: zero


def test_without_a_device():
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    assert _quantize() == 5 and _fp8() == 5
    assert all(_grouped(fn) == 5 for fn in ("", "_dgrad", "_wgrad"))
    x = torch.zeros(4, 128, dtype=torch.bfloat16)
    w = torch.zeros(3, 64, 128, dtype=torch.bfloat16)
    for call in (lambda: B.situ_moe_quantize_fp8_block128(x),
                 lambda: B.situ_moe_matmul_fp8_block128(x.view(torch.uint8), x, w, w),
                 lambda: B.situ_moe_grouped_matmul(x, w), lambda: B.situ_moe_grouped_matmul_dgrad(x, w),
                 lambda: B.situ_moe_grouped_matmul_wgrad(x, x)):
        with pytest.raises(B.SituMoeError) as e:
            call()
        assert e.value.status_name == "SITU_E_DEVICE"


def test_row_division():
    """The multiplier and shift of pairs[r] / div, for every kind of divisor and the largest pairs (the arithmetic of
    the header's make_row_div and the kernel's high product)."""
    for d in list(range(2, 70)) + [127, 128, 129, 1000, 4095, 65536, 99991, (1 << 30) - 1, 1 << 30, (1 << 31) - 1]:
        s = (d - 1).bit_length()
        mul = (1 << (31 + s)) // d + 1
        assert mul < 1 << 32
        for p in (0, 1, d - 1, d, d + 1, 5 * d - 1, 5 * d, (1 << 31) - 1, ((1 << 31) - 1) // d * d,
                  max(((1 << 31) - 1) // d * d - 1, 0)):
            if p < 1 << 31:
                assert ((p * mul) >> 32) >> (s - 1) == p // d, (p, d)


class _Fake:
    """What the binding asks of a device tensor, of any size (its memory is never reached)."""

    def __init__(self, dtype, *shape):
        self.dtype, self.shape, self.is_cuda, self.device = dtype, torch.Size(shape), True, torch.device("cuda", 0)

    def dim(self):
        return len(self.shape)

    def numel(self):
        return self.shape.numel()

    def stride(self):
        return tuple(torch.empty(self.shape, device="meta").stride())

    def is_contiguous(self):
        return True

    def get_device(self):
        return 0

    def data_ptr(self):
        return FAKE


@pytest.fixture
def fakes(monkeypatch):
    if torch.cuda.is_available():
        pytest.skip("a GPU is present: the addresses of these tensors are not memory")
    from block_scaled_mxfp4_amd import grouped
    grouped._first()
    monkeypatch.setattr(grouped, "_device", lambda: 0)
    monkeypatch.setattr(grouped, "_raw_stream", lambda dev: 0)
    return _Fake


def _status(call):
    with pytest.raises(B.SituMoeError) as e:
        call()
    return e.value.status_name


def test_sizes_past_32_bits(fakes):
    """No size loses its upper bits on the way to the library: a call of 2^32 + 128 columns is not one of 128."""
    bf, f32, u8, i32 = torch.bfloat16, torch.float32, torch.uint8, torch.int32
    big = (1 << 32) + 128
    assert _status(lambda: B.situ_moe_quantize_fp8_block128(
        fakes(bf, 1, 128), fakes(u8, 1, 128), fakes(f32, 1, 1))) == "SITU_E_DEVICE"     # the fakes pass where sizes do
    assert _status(lambda: B.situ_moe_quantize_fp8_block128(
        fakes(bf, 1, big), fakes(u8, 1, big), fakes(f32, 1, big // 128))) == "SITU_E_UNSUPPORTED"
    assert _status(lambda: B.situ_moe_matmul_fp8_block128(
        fakes(u8, 1, big), fakes(f32, 1, big // 128), fakes(u8, 8, big), fakes(f32, 1, big // 128),
        out=fakes(bf, 1, 8))) == "SITU_E_UNSUPPORTED"
    x, w, dy = fakes(bf, 4, 128), fakes(bf, 1, 64, 128), fakes(bf, 4, 64)
    pairs, many = fakes(i32, 4), fakes(bf, (1 << 31) + 4, 128)
    for call in (lambda: B.situ_moe_grouped_matmul(x, w, pairs=pairs, x_div=1 << 31, out=dy),
                 lambda: B.situ_moe_grouped_matmul(many, w, pairs=pairs, x_div=1, out=dy),
                 lambda: B.situ_moe_grouped_matmul_dgrad(dy, w, pairs=pairs, dy_div=1 << 31, out=x),
                 lambda: B.situ_moe_grouped_matmul_dgrad(dy, w, pairs=pairs, out_div=1, out=many),
                 lambda: B.situ_moe_grouped_matmul_wgrad(dy, x, pairs=pairs, x_div=1 << 31, out=fakes(f32, 1, 64, 128)),
                 lambda: B.situ_moe_grouped_matmul_wgrad(dy, many, pairs=pairs, x_div=1, out=fakes(f32, 1, 64, 128))):
        assert _status(call) == "SITU_E_UNSUPPORTED"


def test_kernel_of_a_call():
    """The calls of grouped_kernels.py reach the kernels they name on 256 compute units, and all kernels are named."""
    import grouped_kernels as G
    for c in G.CASES:
        product, f32, kernel, counts, n, k, sides = c
        rows, experts = G.rows_of(counts)
        for out in (False, True) if f32 is None else (f32,):
            assert G.kernel_of(product, rows, experts, n, k, f32=out, offsets=not isinstance(counts, int),
                               sides=sides) == kernel, G.case_id(c)
    for product, kernels in G.KERNELS.items():
        assert {c[2] for c in G.CASES if c[0] == product} == {"grouped_" + name for name in kernels}


def test_kernel_of_a_refused_call():
    import grouped_kernels as G
    for args, kw in ((("fwd", 4, 3, 64, 12), {}), (("dgrad", 4, 3, 60, 64), {}), (("fp8", 4, 1, 64, 24), {}),
                     (("fwd", 0, 3, 64, 64), {}), (("fwd", 4, 3, 64, 64), dict(cus=0)),
                     (("fwd", 4, 3, 64, 64), dict(offsets=False)), (("fp8", 0, 1, 64, 64), {})):
        with pytest.raises(B.SituMoeError):
            G.kernel_of(*args, **kw)
    with pytest.raises(B.SituMoeError):
        B.situ_moe_grouped_matmul_kernel(3, B.SituMoeGrouped())
    assert B.load().situ_moe_matmul_fp8_block128_kernel(None, 256) is None
    assert B.load().situ_moe_grouped_matmul_kernel(0, None, 256) is None


def test_kernel_on_any_number_of_units():
    import grouped_kernels as G
    names = {"grouped_" + k for k in G.KERNELS["fwd"]}
    for cus in (1, 8, 304, (1 << 31) - 1):
        for rows, experts, n, k in ((2, 3, 64, 64), (700, 16, 1032, 520), (1 << 24, 1024, 1 << 18, 1 << 18)):
            assert G.kernel_of("fwd", rows, experts, n, k, cus=cus) in names
    assert G.kernel_of("fwd", 2, 3, 64, 64, cus=(1 << 31) - 1) == "grouped_few_kernel 16"   # never enough columns for them
