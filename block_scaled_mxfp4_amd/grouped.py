"""Binding of the FP8 products with scales per 128 and of the bf16 products
with rows grouped by expert (include/situ_moe.h).

As in the rest of the binding nothing here computes on tensor values: the
arguments are checked, outputs that are not given are allocated, and each call
enqueues one kernel on the stream (a torch.cuda.Stream, a raw handle, or None
for the current stream of the tensors' device).  Calls run on the tensors'
device whichever device is current.

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


def _rows(t, name, shape, dtypes, dev):
    """The address and row stride of a matrix whose rows are dense (of any number of rows where shape says None)."""
    if t is None or t.dtype not in dtypes or t.get_device() != dev or t.dim() != 2:
        _bad(t, name, dtypes, dev, f"{shape}, dense rows")
    n, w = t.shape
    stride, one = t.stride()
    if w != shape[1] or (n != shape[0] and shape[0] is not None) or (one != 1 and w > 1):
        _bad(t, name, dtypes, dev, f"{shape}, dense rows")
    return t.data_ptr(), stride if n > 1 else -(-w // 16) * 16   # of one row torch says anything


def _lead(t, name, dtypes, dim):
    """The device of the tensor that says where a call runs, and its shape."""
    if t is None or not t.is_cuda or t.dtype not in dtypes or t.dim() != dim:
        _bad(t, name, dtypes, None, f"{dim} dimensions")
    return t.get_device(), t.shape


class _Place:
    """The device and stream of a call: makes both current while outputs are
    allocated and the kernel is enqueued, where they are not already."""
    __slots__ = ("handle", "entered")

    def __init__(self, dev, stream):
        import torch
        self.entered = ()
        if stream is None and dev == torch.cuda.current_device():
            self.handle = torch._C._cuda_getCurrentRawStream(dev)   # as current_stream(), 2 us sooner
            return
        device = torch.device("cuda", dev)
        if stream is None:
            stream = torch.cuda.current_stream(device)
        elif not isinstance(stream, torch.cuda.Stream):
            stream = torch.cuda.ExternalStream(int(stream), device=device)
        elif stream.device != device:
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


def _out_code(dtype):
    import torch
    if dtype is torch.bfloat16:
        return _B.OUT_BF16
    if dtype is torch.float32:
        return _B.OUT_F32
    _fail(3, f"out_dtype {dtype} (bfloat16 or float32)")


def situ_moe_quantize_fp8_block128(x, codes=None, scales=None, stream=None):
    """E4M3 codes (uint8 [rows, cols]) and fp32 scales ([rows, ceil(cols /
    128)]) of bf16 rows x (a row stride is allowed): scale = max(max |x|,
    2^-100) / 448 per row and 128 columns, code = E4M3 of x / scale, nearest
    even.  cols a multiple of 16.  Returns (codes, scales), allocated here
    when not given."""
    import torch
    dev, (rows, cols) = _lead(x, "x", (torch.bfloat16,), 2)
    xp, stride = _rows(x, "x", (None, cols), (torch.bfloat16,), dev)
    nb = -(-cols // 128)
    with _Place(dev, stream) as handle:
        if codes is None:
            codes = torch.empty(rows, cols, dtype=torch.uint8, device=x.device)
            cp = codes.data_ptr()
        else:
            cp = _dense(codes, "codes", (rows, cols), (torch.uint8, torch.float8_e4m3fn), dev)
        if scales is None:
            scales = torch.empty(rows, nb, dtype=torch.float32, device=x.device)
            sp = scales.data_ptr()
        else:
            sp = _dense(scales, "scales", (rows, nb), (torch.float32,), dev)
        status = _B.load().situ_moe_quantize_fp8_block128(xp, rows, cols, stride, cp, sp, handle)
    if status:
        _B._check(status)
    return codes, scales


def situ_moe_matmul_fp8_block128(a, a_scale, w, w_scale, *, offsets=None, out=None, out_dtype=None, stream=None):
    """out[r, j] = sum over blocks b of 128 along k of a_scale[r, b]
    w_scale[e, j // 128, b] (a w^T over block b), in fp32.

    a: E4M3 codes (uint8 or float8_e4m3fn) [rows, k], a_scale fp32 [rows,
    ceil(k / 128)] (both may have a row stride); w: E4M3 [n, k] with scales
    [ceil(n / 128), ceil(k / 128)], or, grouped, [experts, n, k] with
    [experts, ceil(n / 128), ceil(k / 128)] and offsets int32 [experts + 1]:
    rows offsets[e] .. offsets[e + 1] - 1 belong to expert e.  out: bf16 (the
    default) or fp32 [rows, n]; rows outside every group are left as they are
    (undefined in an output allocated here)."""
    import torch
    types = (torch.uint8, torch.float8_e4m3fn)
    dev, (rows, k) = _lead(a, "a", types, 2)
    ap, a_stride = _rows(a, "a", (rows, k), types, dev)
    kb = -(-k // 128)
    sp, s_stride = _rows(a_scale, "a_scale", (rows, kb), (torch.float32,), dev)
    if offsets is None:
        if w is None or w.dim() != 2:
            _bad(w, "w", types, dev, "[n, k] without offsets")
        n, experts, op = w.shape[0], 1, 0
        wp = _dense(w, "w", (n, k), types, dev)
        wsp = _dense(w_scale, "w_scale", (-(-n // 128), kb), (torch.float32,), dev)
    else:
        if w is None or w.dim() != 3:
            _bad(w, "w", types, dev, "[experts, n, k] with offsets")
        experts, n = w.shape[0], w.shape[1]
        op = _dense(offsets, "offsets", (experts + 1,), (torch.int32,), dev)
        wp = _dense(w, "w", (experts, n, k), types, dev)
        wsp = _dense(w_scale, "w_scale", (experts, -(-n // 128), kb), (torch.float32,), dev)
    with _Place(dev, stream) as handle:
        if out is None:
            out_dtype = out_dtype or torch.bfloat16
            code = _out_code(out_dtype)
            out = torch.empty(rows, n, dtype=out_dtype, device=a.device)
            outp, out_stride = out.data_ptr(), n
        else:
            outp, out_stride = _rows(out, "out", (rows, n), (out_dtype,) if out_dtype else (torch.bfloat16, torch.float32), dev)
            code = _out_code(out.dtype)
        status = _B.load().situ_moe_matmul_fp8_block128(
            _FP8.pack(rows, n, k, experts, code, 0, a_stride, s_stride, out_stride, ap, sp, wp, wsp, op, outp), handle)
    if status:
        _B._check(status)
    return out


def _grouped(name, written, lead, dev, sides, offsets, pairs, divs, sizes, out_dtype, stream):
    """The three grouped products.  sides = (x, y, w) and divs = (x_div,
    y_div); sides[written] is the kernel's output, allocated here if it is
    None; lead: the input whose rows are the positions where pairs is None."""
    import torch
    experts, n, k = sizes
    if offsets is None:
        if experts != 1:
            _fail(1, f"offsets is None with {experts} experts")
        op = 0
    else:
        op = _dense(offsets, "offsets", (experts + 1,), (torch.int32,), dev)
    x_div, y_div = divs
    if pairs is None:
        if x_div or y_div:
            _fail(1, "pairs is None")
        rows, pp = sides[lead].shape[0], 0
    else:
        rows = pairs.numel()
        pp = _dense(pairs, "pairs", (rows,), (torch.int32,), dev)
    shapes = ((None if x_div else rows, k), (None if y_div else rows, n), (experts, n, k))
    names = _NAMES[name]
    with _Place(dev, stream) as handle:
        if sides[written] is None:
            if written < 2 and divs[written]:
                _fail(1, f"{name} with a div on its written side needs out")
            out_dtype = out_dtype or (torch.float32 if written == 2 else torch.bfloat16)
            _out_code(out_dtype)
            out = torch.empty(*shapes[written], dtype=out_dtype, device=sides[lead].device)
            sides = sides[:written] + (out,) + sides[written + 1:]
        either = (out_dtype,) if out_dtype else (torch.bfloat16, torch.float32)
        bf16 = (torch.bfloat16,)
        xp, x_stride = _rows(sides[0], names[0], shapes[0], either if written == 0 else bf16, dev)
        yp, y_stride = _rows(sides[1], names[1], shapes[1], either if written == 1 else bf16, dev)
        wp = _dense(sides[2], names[2], shapes[2], either if written == 2 else bf16, dev)
        out = sides[written]
        status = getattr(_B.load(), name)(
            _GROUPED.pack(rows, n, k, experts, sides[0].shape[0], sides[1].shape[0], x_div, y_div, _out_code(out.dtype),
                          0, x_stride, y_stride, op, pp, xp, yp, wp), handle)
    if status:
        _B._check(status)
    return out


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
    import torch
    dev, _ = _lead(x, "x", (torch.bfloat16,), 2)
    _, sizes = _lead(w, "w", (torch.bfloat16,), 3)
    return _grouped("situ_moe_grouped_matmul", 1, 0, dev, (x, out, w), offsets, pairs, (int(x_div), int(out_div)),
                    sizes, out_dtype, stream)


def situ_moe_grouped_matmul_dgrad(dy, w, offsets=None, *, pairs=None, dy_div=0, out_div=0, out=None, out_dtype=None,
                                  stream=None):
    """The gradient of situ_moe_grouped_matmul in x, one row per position:
    out[o(r)] = w[e]^T dy[i(r)], with i(r) by dy_div and o(r) by out_div (0 or
    1).  A token's gradient is the sum of its pairs' rows.  n and k multiples
    of 8."""
    import torch
    dev, _ = _lead(dy, "dy", (torch.bfloat16,), 2)
    _, sizes = _lead(w, "w", (torch.bfloat16,), 3)
    return _grouped("situ_moe_grouped_matmul_dgrad", 0, 1, dev, (out, dy, w), offsets, pairs,
                    (int(out_div), int(dy_div)), sizes, out_dtype, stream)


def situ_moe_grouped_matmul_wgrad(dy, x, offsets=None, *, pairs=None, dy_div=0, x_div=0, out=None, out_dtype=None,
                                  stream=None):
    """The gradient of situ_moe_grouped_matmul in w: out[e] = sum over the
    positions of e of dy[i(r)] x[j(r)]^T, [experts, n, k] in fp32 (the
    default) or bf16; zero for an empty expert.  i(r) by dy_div, j(r) by
    x_div.  n and k multiples of 8."""
    import torch
    dev, (_, n) = _lead(dy, "dy", (torch.bfloat16,), 2)
    _, (_, k) = _lead(x, "x", (torch.bfloat16,), 2)
    experts = 1 if offsets is None else offsets.numel() - 1
    return _grouped("situ_moe_grouped_matmul_wgrad", 2, 1 if dy_div == 0 else 0, dev, (x, dy, out), offsets, pairs,
                    (int(x_div), int(dy_div)), (experts, n, k), out_dtype, stream)
