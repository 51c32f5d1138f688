"""Binding of the FP8 products with scales per 128 and of the bf16 products
with rows grouped by expert (include/situ_moe.h).

As in the rest of the binding nothing here computes on tensor values: the
arguments are checked, outputs that are not given are allocated, and each call
enqueues one kernel on the stream (a torch.cuda.Stream, a raw handle, or None
for the current stream of the tensors' device).  Calls run on the tensors'
device whichever device is current.
"""

import ctypes

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


def _fail(status, message):
    raise _B.SituMoeError(status, message)


def _tensor(t, name, dtypes, dim, device=None):
    if t is None:
        _fail(1, f"{name} is None")
    if not t.is_cuda:
        _fail(5, f"{name} must be a device tensor")
    if device is not None and t.device != device:
        _fail(2, f"{name} is on {t.device}, not {device}")
    if t.dtype not in dtypes:
        _fail(2, f"{name} has dtype {t.dtype}, expected {' or '.join(map(str, dtypes))}")
    if t.dim() != dim:
        _fail(2, f"{name} has {t.dim()} dimensions, expected {dim}")


def _row_stride(t, name):
    """Elements between the rows of a matrix whose rows are dense."""
    rows, cols = t.shape
    if cols > 1 and t.stride(1) != 1:
        _fail(2, f"the rows of {name} must be dense")
    return t.stride(0) if rows > 1 else -(-cols // 16) * 16


def _dense(t, name, shape, dtypes, device):
    _tensor(t, name, dtypes, len(shape), device)
    if tuple(t.shape) != tuple(shape):
        _fail(2, f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if not t.is_contiguous():
        _fail(2, f"{name} must be contiguous")


def _out_code(out_dtype):
    import torch
    if out_dtype == torch.bfloat16:
        return _B.OUT_BF16
    if out_dtype == torch.float32:
        return _B.OUT_F32
    _fail(3, f"out_dtype {out_dtype} (bfloat16 or float32)")


class _Place:
    """The device and stream of a call: makes both current while outputs are
    allocated and the kernel is enqueued, where they are not already."""
    __slots__ = ("handle", "entered")

    def __init__(self, device, stream):
        import torch
        self.entered = ()
        if stream is None and device.index == torch.cuda.current_device():
            self.handle = torch._C._cuda_getCurrentRawStream(device.index)   # as current_stream(), 2 us sooner
            return
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


def situ_moe_quantize_fp8_block128(x, codes=None, scales=None, stream=None):
    """E4M3 codes (uint8 [rows, cols]) and fp32 scales ([rows, ceil(cols /
    128)]) of bf16 rows x (a row stride is allowed): scale = max(max |x|,
    2^-100) / 448 per row and 128 columns, code = E4M3 of x / scale, nearest
    even.  cols a multiple of 16.  Returns (codes, scales), allocated here
    when not given."""
    import torch
    _tensor(x, "x", (torch.bfloat16,), 2)
    rows, cols = x.shape
    stride = _row_stride(x, "x")
    with _Place(x.device, stream) as handle:
        if codes is None:
            codes = torch.empty((rows, cols), dtype=torch.uint8, device=x.device)
        else:
            _dense(codes, "codes", (rows, cols), (torch.uint8, torch.float8_e4m3fn), x.device)
        if scales is None:
            scales = torch.empty((rows, -(-cols // 128)), dtype=torch.float32, device=x.device)
        else:
            _dense(scales, "scales", (rows, -(-cols // 128)), (torch.float32,), x.device)
        _B._check(_B.load().situ_moe_quantize_fp8_block128(x.data_ptr(), rows, cols, stride, codes.data_ptr(),
                                                           scales.data_ptr(), handle))
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
    codes = (torch.uint8, torch.float8_e4m3fn)
    _tensor(a, "a", codes, 2)
    dev = a.device
    rows, k = a.shape
    _tensor(w, "w", codes, 2 if offsets is None else 3, dev)
    n = w.shape[-2]
    experts = 1 if offsets is None else w.shape[0]
    nb, kb = -(-n // 128), -(-k // 128)
    lead = () if offsets is None else (experts,)
    _dense(w, "w", lead + (n, k), codes, dev)
    _dense(w_scale, "w_scale", lead + (nb, kb), (torch.float32,), dev)
    _tensor(a_scale, "a_scale", (torch.float32,), 2, dev)
    if tuple(a_scale.shape) != (rows, kb):
        _fail(2, f"a_scale has shape {tuple(a_scale.shape)}, expected {(rows, kb)}")
    if offsets is not None:
        _dense(offsets, "offsets", (experts + 1,), (torch.int32,), dev)
    with _Place(dev, stream) as handle:
        if out is None:
            out = torch.empty((rows, n), dtype=out_dtype or torch.bfloat16, device=dev)
        else:
            _tensor(out, "out", (out_dtype,) if out_dtype else (torch.bfloat16, torch.float32), 2, dev)
            if tuple(out.shape) != (rows, n):
                _fail(2, f"out has shape {tuple(out.shape)}, expected {(rows, n)}")
        args = SituMoeFp8Matmul(rows, n, k, experts, _out_code(out.dtype), 0, _row_stride(a, "a"),
                                _row_stride(a_scale, "a_scale"), _row_stride(out, "out"), a.data_ptr(),
                                a_scale.data_ptr(), w.data_ptr(), w_scale.data_ptr(),
                                None if offsets is None else offsets.data_ptr(), out.data_ptr())
        _B._check(_B.load().situ_moe_matmul_fp8_block128(ctypes.byref(args), handle))
    return out


def _grouped(name, written, x, y, w, offsets, pairs, x_div, y_div, sizes, out_dtype, stream):
    """The three grouped products: `written` names the side (x, y or w) the
    kernel writes, which is allocated here if it is None; sizes = (experts,
    n, k)."""
    import torch
    sides = {"x": x, "y": y, "w": w}
    read = "y" if written == "x" else "x"
    _tensor(sides[read], _NAMES[name][read], (torch.bfloat16,), 2)
    dev = sides[read].device
    experts, n, k = sizes
    if offsets is None and experts != 1:
        _fail(1, f"offsets is None with {experts} experts")
    if offsets is not None:
        _dense(offsets, "offsets", (experts + 1,), (torch.int32,), dev)
    x_div, y_div = int(x_div), int(y_div)
    if pairs is not None:
        _tensor(pairs, "pairs", (torch.int32,), 1, dev)
        if not pairs.is_contiguous():
            _fail(2, "pairs must be contiguous")
        rows = pairs.shape[0]
    else:
        if x_div or y_div:
            _fail(1, "pairs is None")
        rows = sides[read].shape[0]
    with _Place(dev, stream) as handle:
        if sides[written] is None:
            shape = {"x": (rows, k), "y": (rows, n), "w": (experts, n, k)}[written]
            if written != "w" and (x_div if written == "x" else y_div):
                _fail(1, f"{name} with a div on its written side needs `out`")
            sides[written] = torch.empty(shape, dtype=out_dtype, device=dev)
        out = sides[written]
        either = (out_dtype,) if out_dtype is not None else (torch.bfloat16, torch.float32)
        for s, width, div in (("x", k, x_div), ("y", n, y_div)):
            t, label = sides[s], "out" if s == written else _NAMES[name][s]
            _tensor(t, label, either if s == written else (torch.bfloat16,), 2, dev)
            if t.shape[1] != width or (not div and t.shape[0] != rows):
                _fail(2, f"{label} has shape {tuple(t.shape)}, expected {(t.shape[0] if div else rows, width)}")
        _dense(sides["w"], "out" if written == "w" else "w", (experts, n, k),
               either if written == "w" else (torch.bfloat16,), dev)
        x, y, w = sides["x"], sides["y"], sides["w"]
        args = SituMoeGrouped(rows, n, k, experts, x.shape[0], y.shape[0], x_div, y_div, _out_code(out.dtype), 0,
                              _row_stride(x, "x"), _row_stride(y, "y"),
                              None if offsets is None else offsets.data_ptr(),
                              None if pairs is None else pairs.data_ptr(), x.data_ptr(), y.data_ptr(), w.data_ptr())
        _B._check(getattr(_B.load(), name)(ctypes.byref(args), handle))
    return out


_NAMES = {"situ_moe_grouped_matmul": {"x": "x"}, "situ_moe_grouped_matmul_dgrad": {"y": "dy"},
          "situ_moe_grouped_matmul_wgrad": {"x": "x", "y": "dy"}}


def _weights(w):
    import torch
    _tensor(w, "w", (torch.bfloat16,), 3)
    return tuple(w.shape)


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
    if out is None:
        out_dtype = out_dtype or torch.bfloat16
    return _grouped("situ_moe_grouped_matmul", "y", x, out, w, offsets, pairs, x_div, out_div, _weights(w), out_dtype,
                    stream)


def situ_moe_grouped_matmul_dgrad(dy, w, offsets=None, *, pairs=None, dy_div=0, out_div=0, out=None, out_dtype=None,
                                  stream=None):
    """The gradient of situ_moe_grouped_matmul in x, one row per position:
    out[o(r)] = w[e]^T dy[i(r)], with i(r) by dy_div and o(r) by out_div (0 or
    1).  A token's gradient is the sum of its pairs' rows.  n and k multiples
    of 8."""
    import torch
    if out is None:
        out_dtype = out_dtype or torch.bfloat16
    return _grouped("situ_moe_grouped_matmul_dgrad", "x", out, dy, w, offsets, pairs, out_div, dy_div, _weights(w),
                    out_dtype, stream)


def situ_moe_grouped_matmul_wgrad(dy, x, offsets=None, *, pairs=None, dy_div=0, x_div=0, out=None, out_dtype=None,
                                  stream=None):
    """The gradient of situ_moe_grouped_matmul in w: out[e] = sum over the
    positions of e of dy[i(r)] x[j(r)]^T, [experts, n, k] in fp32 (the
    default) or bf16; zero for an empty expert.  i(r) by dy_div, j(r) by
    x_div.  n and k multiples of 8."""
    import torch
    _tensor(dy, "dy", (torch.bfloat16,), 2)
    _tensor(x, "x", (torch.bfloat16,), 2)
    if out is None:
        out_dtype = out_dtype or torch.float32
    experts = 1 if offsets is None else offsets.numel() - 1
    return _grouped("situ_moe_grouped_matmul_wgrad", "w", x, dy, out, offsets, pairs, x_div, dy_div,
                    (experts, dy.shape[1], x.shape[1]), out_dtype, stream)
