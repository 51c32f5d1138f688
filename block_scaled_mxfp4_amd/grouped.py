"""Binding of the FP8 products with scales per 128 and of the bf16 products
with rows grouped by expert (include/situ_moe.h).

As in the rest of the binding nothing here computes on tensor values: the
arguments are checked, outputs that are not given are allocated, and each call
enqueues one kernel on the stream (a torch.cuda.Stream, a raw handle, or None
for the current stream of the tensors' device).  Calls run on the tensors'
device whichever device is current.  An output carries no autograd graph,
whether or not an input requires grad: a caller who trains calls the _dgrad and
_wgrad products.

A decode-sized call costs more on the host than on the GPU, so the checks test
what a right argument has in one expression and look for the reason only when
that fails, and the argument structs are packed rather than built by field.
"""

import ctypes
import struct

import block_scaled_mxfp4_amd as _B


class SituMoeFp8Matmul(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("rows", "n", "k", "experts", "out_dtype", "reserved")] + \
               [(n, ctypes.c_int64) for n in ("a_stride", "a_scale_stride", "out_stride")] + \
               [(n, ctypes.c_void_p) for n in ("a", "a_scale", "w", "w_scale", "offsets", "out")]


class SituMoeGrouped(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("rows", "n", "k", "experts", "x_rows", "y_rows", "x_div", "y_div",
                                              "out_dtype", "reserved")] + \
               [(n, ctypes.c_int64) for n in ("x_stride", "y_stride")] + \
               [(n, ctypes.c_void_p) for n in ("offsets", "pairs", "x", "y", "w")]


_FP8 = struct.Struct("=6i3q6Q")
_GROUPED = struct.Struct("=10i2q5Q")
assert _FP8.size == ctypes.sizeof(SituMoeFp8Matmul) and _GROUPED.size == ctypes.sizeof(SituMoeGrouped)


def _pack(form, *fields):
    try:
        return form.pack(*fields)
    except struct.error:
        _fail(3, "a size or div past 32 bits")


# torch and what the calls use of it, looked up once: importing this package imports neither torch nor the library
torch = _device = _raw_stream = _empty = _library = None
_BF16 = _F32 = _EITHER = _CODES = _INT32 = ()


def _first():
    global torch, _device, _raw_stream, _empty, _library, _BF16, _F32, _EITHER, _CODES, _INT32
    import torch as t
    _library = _B.load()
    _device, _raw_stream, _empty = t._C._cuda_getDevice, t._C._cuda_getCurrentRawStream, t.empty
    _BF16, _F32, _EITHER = (t.bfloat16,), (t.float32,), (t.bfloat16, t.float32)
    _CODES, _INT32 = (t.uint8, t.float8_e4m3fn), (t.int32,)
    torch = t


def _fail(status, message):
    raise _B.SituMoeError(status, message)


def _bad(t, name, dtypes, dev, want):
    """The reason why t is refused."""
    if t is None:
        _fail(1, f"{name} is None")
    if not t.is_cuda:
        _fail(5, f"{name} must be a device tensor")
    if dev is not None and t.get_device() != dev:
        _fail(2, f"{name} is on {t.device}, not device {dev}")
    if t.dtype not in dtypes:
        _fail(2, f"{name} has dtype {t.dtype}, expected {' or '.join(map(str, dtypes))}")
    _fail(2, f"{name} has shape {tuple(t.shape)}, strides {t.stride()}; expected {want}")


def _dense(t, name, shape, dtypes, dev):
    """The address of a contiguous tensor."""
    if t is None or t.dtype not in dtypes or t.get_device() != dev or t.shape != shape or not t.is_contiguous():
        _bad(t, name, dtypes, dev, f"{shape}, contiguous")
    return t.data_ptr()


def _lead(t, name, dtypes):
    """Device, rows, columns, row stride and address of the matrix that says where a call runs."""
    if t is None or not t.is_cuda or t.dtype not in dtypes or t.dim() != 2:
        _bad(t, name, dtypes, None, "a matrix")
    n, w = t.shape
    stride, one = t.stride()
    if one != 1 and w > 1:
        _bad(t, name, dtypes, None, "dense rows")
    return t.get_device(), n, w, stride if n > 1 else -(-w // 16) * 16, t.data_ptr()   # of one row torch says anything


def _rows(t, name, n, w, dtypes, dev):
    """Rows, row stride and address of a matrix [n, w] whose rows are dense (any number of them where n is None)."""
    if t is None or t.dtype not in dtypes or t.get_device() != dev or t.dim() != 2:
        _bad(t, name, dtypes, dev, f"({n}, {w}), dense rows")
    m, v = t.shape
    stride, one = t.stride()
    if v != w or (m != n and n is not None) or (one != 1 and w > 1):
        _bad(t, name, dtypes, dev, f"({n}, {w}), dense rows")
    return m, stride if m > 1 else -(-w // 16) * 16, t.data_ptr()


class _Place:
    """The device and stream of a call: makes both current while outputs are
    allocated and the kernel is enqueued, where they are not already."""

    def __init__(self, dev, stream):
        device = torch.device("cuda", dev)
        stream = _B._torch_stream(stream, device)
        if stream.device != device:
            _fail(2, f"the stream is of {stream.device}, the tensors are on {device}")
        self.handle = stream.cuda_stream
        self.entered = (torch.cuda.device(device), torch.cuda.stream(stream))

    def __enter__(self):
        for c in self.entered:
            c.__enter__()
        return self.handle

    def __exit__(self, *e):
        for c in reversed(self.entered):
            c.__exit__(*e)


def _at(dev, stream, call, *args):
    """call(handle, *args) on the device and stream."""
    if stream is None and dev == _device():
        return call(_raw_stream(dev), *args)
    with _Place(dev, stream) as handle:
        return call(handle, *args)


def _out_code(dtype):
    if dtype is torch.bfloat16:
        return _B.OUT_BF16
    if dtype is torch.float32:
        return _B.OUT_F32
    _fail(3, f"out_dtype {dtype} (bfloat16 or float32)")


def _out_types(out_dtype):
    return _EITHER if out_dtype is None else (out_dtype,)


def situ_moe_quantize_fp8_block128(x, codes=None, scales=None, stream=None):
    """E4M3 codes (uint8 [rows, cols]) and fp32 scales ([rows, ceil(cols /
    128)]) of bf16 rows x (a row stride is allowed): scale = max(max |x|,
    2^-100) / 448 per row and 128 columns, code = E4M3 of x / scale, nearest
    even.  cols a multiple of 16.  Returns (codes, scales), allocated here
    when not given."""
    if torch is None:
        _first()
    dev, rows, cols, stride, xp = _lead(x, "x", _BF16)
    return _at(dev, stream, _quantize, x.device, dev, rows, cols, stride, xp, codes, scales)


def _quantize(handle, device, dev, rows, cols, stride, xp, codes, scales):
    if cols >= 1 << 31:                    # ctypes would pass its low 32 bits
        _fail(3, f"cols {cols} past 32 bits")
    nb = -(-cols // 128)
    if codes is None:
        codes = _empty(rows, cols, dtype=torch.uint8, device=device)
        cp = codes.data_ptr()
    else:
        cp = _dense(codes, "codes", (rows, cols), _CODES, dev)
    if scales is None:
        scales = _empty(rows, nb, dtype=torch.float32, device=device)
        sp = scales.data_ptr()
    else:
        sp = _dense(scales, "scales", (rows, nb), _F32, dev)
    status = _library.situ_moe_quantize_fp8_block128(xp, rows, cols, stride, cp, sp, handle)
    if status:
        _B._check(status)
    return codes, scales


def situ_moe_matmul_fp8_block128(a, a_scale, w, w_scale, *, offsets=None, out=None, out_dtype=None, stream=None):
    """out[r, j] = sum over blocks b of 128 along k of a_scale[r, b]
    w_scale[e, j // 128, b] (a w^T over block b).  An fp32 output is an fp32
    sum.  A bf16 output of more than a few rows sums each block by the FP8
    matrix instruction, which drops from the products of each aligned eight
    elements of k what lies 13 bits below the largest one's leading bit: off by
    at most 7 * 2^-13 of the largest scaled product of each eight, summed, and
    then rounded to bf16.  Where large products cancel that is more than the
    rounding; out_dtype=torch.float32 has no such loss.

    a: E4M3 codes (uint8 or float8_e4m3fn) [rows, k], a_scale fp32 [rows,
    ceil(k / 128)] (both may have a row stride); w: E4M3 [n, k] with scales
    [ceil(n / 128), ceil(k / 128)], or, grouped, [experts, n, k] with
    [experts, ceil(n / 128), ceil(k / 128)] and offsets int32 [experts + 1]:
    rows offsets[e] .. offsets[e + 1] - 1 belong to expert e.  out: bf16 (the
    default) or fp32 [rows, n]; rows outside every group are left as they are
    (undefined in an output allocated here)."""
    if torch is None:
        _first()
    dev, rows, k, a_stride, ap = _lead(a, "a", _CODES)
    kb = -(-k // 128)
    _, s_stride, sp = _rows(a_scale, "a_scale", rows, kb, _F32, dev)
    if offsets is None:
        if w is None or w.dim() != 2:
            _bad(w, "w", _CODES, dev, "[n, k] without offsets")
        n, experts, op = w.shape[0], 1, 0
        wp = _dense(w, "w", (n, k), _CODES, dev)
        wsp = _dense(w_scale, "w_scale", (-(-n // 128), kb), _F32, dev)
    else:
        if w is None or w.dim() != 3:
            _bad(w, "w", _CODES, dev, "[experts, n, k] with offsets")
        experts, n, _ = w.shape
        op = _dense(offsets, "offsets", (experts + 1,), _INT32, dev)
        wp = _dense(w, "w", (experts, n, k), _CODES, dev)
        wsp = _dense(w_scale, "w_scale", (experts, -(-n // 128), kb), _F32, dev)
    return _at(dev, stream, _matmul, a.device, dev, (rows, n, k, experts), (a_stride, s_stride), (ap, sp, wp, wsp, op),
               out, out_dtype)


def _matmul(handle, device, dev, sizes, strides, pointers, out, out_dtype):
    rows, n = sizes[:2]
    if out is None:
        out_dtype = out_dtype or torch.bfloat16
        code = _out_code(out_dtype)
        out = _empty(rows, n, dtype=out_dtype, device=device)
        stride, outp = n, out.data_ptr()
    else:
        _, stride, outp = _rows(out, "out", rows, n, _out_types(out_dtype), dev)
        code = _out_code(out.dtype)
    status = _library.situ_moe_matmul_fp8_block128(_pack(_FP8, *sizes, code, 0, *strides, stride, *pointers, outp),
                                                   handle)
    if status:
        _B._check(status)
    return out


def _grouped(handle, name, written, lead, device, dev, sides, offsets, pairs, x_div, y_div, experts, n, k, out_dtype):
    """The three grouped products.  sides = [x, y, w]; sides[written] is the
    kernel's output, allocated here if it is None; lead: the input whose rows
    are the positions where pairs is None."""
    if offsets is None:
        if experts != 1:
            _fail(1, f"offsets is None with {experts} experts")
        op = 0
    else:
        op = _dense(offsets, "offsets", (experts + 1,), _INT32, dev)
    if pairs is None:
        if x_div or y_div:
            _fail(1, "pairs is None")
        rows, pp = sides[lead].shape[0], 0
    else:
        rows = pairs.numel()
        pp = _dense(pairs, "pairs", (rows,), _INT32, dev)
    names = _NAMES[name]
    out = sides[written]
    types = _out_types(out_dtype)
    if out is None:
        if written < 2 and (y_div if written else x_div):
            _fail(1, f"{name} with a div on its written side needs out")
        if out_dtype is None:
            out_dtype = torch.float32 if written == 2 else torch.bfloat16
        code = _out_code(out_dtype)
        types = (out_dtype,)
        if written == 2:
            out = _empty(experts, n, k, dtype=out_dtype, device=device)
        else:
            out = _empty(rows, n if written else k, dtype=out_dtype, device=device)
        sides[written] = out
    x, y, w = sides
    x_rows, x_stride, xp = _rows(x, names[0], None if x_div else rows, k, types if written == 0 else _BF16, dev)
    y_rows, y_stride, yp = _rows(y, names[1], None if y_div else rows, n, types if written == 1 else _BF16, dev)
    wp = _dense(w, names[2], (experts, n, k), types if written == 2 else _BF16, dev)
    status = getattr(_library, name)(
        _pack(_GROUPED, rows, n, k, experts, x_rows, y_rows, x_div, y_div, _out_code(out.dtype), 0, x_stride, y_stride, op,
              pp, xp, yp, wp), handle)
    if status:
        _B._check(status)
    return out


def _weights(w):
    if w is None or not w.is_cuda or w.dtype not in _BF16 or w.dim() != 3:
        _bad(w, "w", _BF16, None, "[experts, n, k]")
    return w.shape


_NAMES = {"situ_moe_grouped_matmul": ("x", "out", "w"), "situ_moe_grouped_matmul_dgrad": ("out", "dy", "w"),
          "situ_moe_grouped_matmul_wgrad": ("x", "dy", "out")}


def situ_moe_grouped_matmul(x, w, offsets=None, *, pairs=None, x_div=0, out_div=0, out=None, out_dtype=None,
                            stream=None):
    """out[o(r)] = w[e] x[i(r)] for the positions r = offsets[e] ..
    offsets[e + 1] - 1 of each expert e.

    x: bf16 [x_rows, k]; w: bf16 [experts, n, k]; offsets: int32 [experts + 1]
    (None with one expert: all positions).  i(r) = r with x_div = 0, else
    pairs[r] // x_div; o(r) likewise with out_div (0 or 1).  pairs: int32
    [positions].  k a multiple of 8.  out: bf16 (the default) or fp32; rows no
    position stands for are left as they are (undefined in an output allocated
    here); with out_div = 1 it has to be given."""
    if torch is None:
        _first()
    if x is None or not x.is_cuda or x.dim() != 2:
        _bad(x, "x", _BF16, None, "a matrix")
    dev = x.get_device()
    return _at(dev, stream, _grouped, "situ_moe_grouped_matmul", 1, 0, x.device, dev, [x, out, w], offsets, pairs,
               int(x_div), int(out_div), *_weights(w), out_dtype)


def situ_moe_grouped_matmul_dgrad(dy, w, offsets=None, *, pairs=None, dy_div=0, out_div=0, out=None, out_dtype=None,
                                  stream=None):
    """The gradient of situ_moe_grouped_matmul in x, one row per position:
    out[o(r)] = w[e]^T dy[i(r)], with i(r) by dy_div and o(r) by out_div (0 or
    1).  A token's gradient is the sum of its pairs' rows.  n and k multiples
    of 8."""
    if torch is None:
        _first()
    if dy is None or not dy.is_cuda or dy.dim() != 2:
        _bad(dy, "dy", _BF16, None, "a matrix")
    dev = dy.get_device()
    return _at(dev, stream, _grouped, "situ_moe_grouped_matmul_dgrad", 0, 1, dy.device, dev, [out, dy, w], offsets, pairs,
               int(out_div), int(dy_div), *_weights(w), out_dtype)


def situ_moe_grouped_matmul_wgrad(dy, x, offsets=None, *, pairs=None, dy_div=0, x_div=0, out=None, out_dtype=None,
                                  stream=None):
    """The gradient of situ_moe_grouped_matmul in w: out[e] = sum over the
    positions of e of dy[i(r)] x[j(r)]^T, [experts, n, k] in fp32 (the
    default) or bf16; zero for an empty expert.  i(r) by dy_div, j(r) by
    x_div.  n and k multiples of 8."""
    if torch is None:
        _first()
    dev, _, n, _, _ = _lead(dy, "dy", _BF16)
    _, _, k, _, _ = _lead(x, "x", _BF16)
    experts = 1 if offsets is None else max(offsets.numel() - 1, 0)
    return _at(dev, stream, _grouped, "situ_moe_grouped_matmul_wgrad", 2, 0 if dy_div else 1, dy.device, dev, [x, dy, out],
               offsets, pairs, int(x_div), int(dy_div), experts, n, k, out_dtype)


def _name(kernel):
    if kernel is None:
        raise _B.SituMoeError(2, _B.situ_moe_last_error())
    return kernel.decode()


def situ_moe_matmul_fp8_block128_kernel(args, cus=256):
    """The kernel that a SituMoeFp8Matmul is given to on a device of `cus`
    compute units; nothing is launched and its addresses are not followed."""
    return _name(_B.load().situ_moe_matmul_fp8_block128_kernel(ctypes.byref(args), cus))


def situ_moe_grouped_matmul_kernel(direction, args, cus=256):
    """The same of a SituMoeGrouped.  direction: 0 the product, 1 dgrad, 2 wgrad."""
    return _name(_B.load().situ_moe_grouped_matmul_kernel(direction, ctypes.byref(args), cus))
