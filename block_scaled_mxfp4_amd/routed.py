"""Binding of the steps around the routed products: the gate with its balance
loss, the gated activation with gate and up kept in 8 bits, the combine, the
gradients of the three, and the adapters of many requests beside a shared
projection (include/situ_moe.h).

As in grouped.py: the arguments are checked, outputs that are not given are
allocated on the call's stream, and the kernels are enqueued on the tensors'
device; nothing here computes on tensor values, and no output carries an
autograd graph.
"""

import ctypes
import functools
import struct

import block_scaled_mxfp4_amd as _B
from . import grouped as _G
from .grouped import _Place, _bad, _dense, _fail, _lead, _out_code, _rows

SCORINGS = {"softmax": 0, "sigmoid": 1}


class SituMoeRouter(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("tokens", "experts", "top_k", "scoring", "logits_dtype", "weights_dtype",
                                              "renormalize")] + \
               [("scale", ctypes.c_float), ("logits_stride", ctypes.c_int64)] + \
               [(n, ctypes.c_void_p) for n in ("logits", "bias", "mask", "ids", "weights", "packed", "counts",
                                               "prob_sum", "loss", "workspace")] + \
               [("workspace_bytes", ctypes.c_uint64)]


class SituMoeRouterBackward(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("tokens", "experts", "top_k", "scoring", "logits_dtype", "out_dtype",
                                              "renormalize")] + \
               [("scale", ctypes.c_float)] + [(n, ctypes.c_int64) for n in ("logits_stride", "out_stride")] + \
               [(n, ctypes.c_void_p) for n in ("logits", "mask", "ids", "d_weights", "counts", "d_loss", "d_logits")]


class SituMoeActivation(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("rows", "inner", "experts", "activation")] + \
               [(n, ctypes.c_int64) for n in ("gate_up_stride", "h_stride", "dh_stride", "d_gate_up_stride")] + \
               [(n, ctypes.c_void_p) for n in ("offsets", "p0", "p1", "gate_up", "h", "codes", "scales", "dh",
                                               "d_gate_up")]


class SituMoeCombine(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("tokens", "top_k", "hidden", "rows", "y_dtype", "weights_dtype",
                                              "out_dtype", "reserved")] + \
               [(n, ctypes.c_int64) for n in ("y_stride", "out_stride", "dy_stride")] + \
               [(n, ctypes.c_void_p) for n in ("y", "weights", "inv", "out", "dy", "d_weights")]


class SituMoeAdapters(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("rows", "n", "k", "rank", "requests", "adapters", "out_dtype",
                                              "reserved")] + \
               [(n, ctypes.c_int64) for n in ("x_stride", "base_stride", "out_stride")] + \
               [(n, ctypes.c_void_p) for n in ("offsets", "adapter", "ranks", "scales", "x", "a", "b", "base", "out",
                                               "workspace")] + \
               [("workspace_bytes", ctypes.c_uint64)]


_ROUTER, _ROUTER_BACKWARD = struct.Struct("=7ifq10QQ"), struct.Struct("=7if2q7Q")
_ACTIVATION, _COMBINE, _ADAPTERS = struct.Struct("=4i4q9Q"), struct.Struct("=8i3q6Q"), struct.Struct("=8i3q10QQ")
assert all(s.size == ctypes.sizeof(c) for s, c in (
    (_ROUTER, SituMoeRouter), (_ROUTER_BACKWARD, SituMoeRouterBackward), (_ACTIVATION, SituMoeActivation),
    (_COMBINE, SituMoeCombine), (_ADAPTERS, SituMoeAdapters)))


# looked up once, as grouped.py does: importing this package imports neither torch nor the library
torch = _device = _raw_stream = _empty = _library = None
_BF16 = _F32 = _EITHER = _CODES = _INT32 = _MASK = ()


def _first():
    global torch, _device, _raw_stream, _empty, _library, _BF16, _F32, _EITHER, _CODES, _INT32, _MASK
    if _G.torch is None:
        _G._first()
    _device, _raw_stream, _empty, _library = _G._device, _G._raw_stream, _G._empty, _G._library
    _BF16, _F32, _EITHER, _CODES, _INT32 = _G._BF16, _G._F32, _G._EITHER, _G._CODES, _G._INT32
    _MASK = (_G.torch.bool, _G.torch.uint8)
    torch = _G.torch


def _elsewhere(dev, stream, call, *args):
    """call(handle, *args) on a device or stream that is not the current one."""
    with _Place(dev, stream) as handle:
        return call(handle, *args)


def _pack(form, *fields):
    try:
        return form.pack(*fields)
    except (struct.error, OverflowError):
        _fail(3, "a size past 32 bits, or a scale past fp32")


def _run(entry, handle, form, *fields):
    status = entry(_pack(form, *fields), handle)
    if status:
        _B._check(status)


def _need_bytes(fn, args):
    n = ctypes.c_uint64()
    _B._check(fn(args, ctypes.byref(n)))
    return n.value


@functools.lru_cache(maxsize=256)
def _router_bytes(tokens, experts):
    return _need_bytes(_library.situ_moe_router_workspace,
                       _pack(_ROUTER, tokens, experts, 1, 0, 0, 0, 0, 1.0, 0, *[0] * 6, 1, 1, 1, 0, 0))


@functools.lru_cache(maxsize=256)
def _adapters_bytes(rows, n, k, rank, requests):
    return _need_bytes(_library.situ_moe_adapters_workspace,
                       _pack(_ADAPTERS, rows, n, k, rank, requests, *[0] * 6, *[0] * 11))


def _workspace(given, need, device, dev):
    """Address and bytes of a workspace, and the tensor that holds them."""
    if not need:
        return 0, 0, given
    if given is None:
        given = _empty(need, dtype=torch.uint8, device=device)
        return given.data_ptr(), need, given
    if given.get_device() != dev or not given.is_contiguous():
        _bad(given, "workspace", (given.dtype,), dev, "contiguous")
    return given.data_ptr(), given.numel() * given.element_size(), given


def _maybe(t, name, shape, dtypes, dev):
    return 0 if t is None else _dense(t, name, shape, dtypes, dev)


def _made(t, name, shape, dtype, device, dev):
    """An output and its address, allocated here if it is None."""
    if t is None:
        t = _empty(*shape, dtype=dtype, device=device)
        return t, t.data_ptr()
    return t, _dense(t, name, shape, (dtype,), dev)


def _scoring(name):
    code = SCORINGS.get(name)
    return _fail(3, f"scoring {name!r} (softmax or sigmoid)") if code is None else code


def situ_moe_router(logits, top_k, *, scoring="softmax", bias=None, renormalize=True, scale=1.0, mask=None,
                    balance=False, packed=None, ids=None, weights=None, weights_dtype=None, counts=None, prob_sum=None,
                    loss=None, workspace=None, stream=None):
    """Expert ids (int32 [tokens, top_k], in descending order of score) and
    weights (bf16, or weights_dtype) of each token from logits [tokens,
    experts] (fp32 or bf16; a row stride is allowed).

    scoring: softmax over the experts or sigmoid; bias (fp32 [experts], sigmoid
    only) is added for the choice alone; among equals the lowest id.  weights =
    scale * score, divided by the sum of the chosen scores with renormalize.
    mask (bool or uint8 [tokens]): rows of 0 are not routed: ids -1, weights 0.
    Experts whose logit is -inf or NaN are never chosen (id -1, weight 0 where
    none is left).

    packed=True (or an int32 [tokens, top_k] tensor) also gives the layer's
    topk_packed.  balance=True (or counts, prob_sum and loss given) also gives
    counts int32 [experts], prob_sum fp32 [experts] and the balance loss fp32 [1],
        experts * top_k / C^2 * sum_e counts[e] prob_sum[e],  C = sum counts.

    Returns (ids, weights[, packed][, counts, prob_sum, loss])."""
    if torch is None:
        _first()
    dev, tokens, experts, stride, lp = _lead(logits, "logits", _EITHER)
    args = (logits, dev, tokens, experts, stride, lp, int(top_k), _scoring(scoring), bias, bool(renormalize), scale,
            mask, balance, packed, ids, weights, weights_dtype, counts, prob_sum, loss, workspace)
    if stream is None and dev == _device():
        return _router(_raw_stream(dev), *args)
    return _elsewhere(dev, stream, _router, *args)


def _router(handle, logits, dev, tokens, experts, stride, lp, top_k, scoring, bias, renormalize, scale, mask, balance,
            packed, ids, weights, weights_dtype, counts, prob_sum, loss, workspace):
    device = logits.device
    if not 0 < top_k <= experts:
        _fail(2, f"top_k {top_k} of {experts} experts")
    shape = (tokens, top_k)
    ids, ip = _made(ids, "ids", shape, torch.int32, device, dev)
    if weights_dtype is None:
        weights_dtype = torch.bfloat16 if weights is None else weights.dtype
    code = _out_code(weights_dtype)
    weights, wp = _made(weights, "weights", shape, weights_dtype, device, dev)
    out = (ids, weights)
    pp = 0
    if packed is not None and packed is not False:
        packed, pp = _made(None if packed is True else packed, "packed", shape, torch.int32, device, dev)
        out += (packed,)
    cp = sp = op = wsp = need = 0
    if balance or counts is not None or prob_sum is not None or loss is not None:
        counts, cp = _made(counts, "counts", (experts,), torch.int32, device, dev)
        prob_sum, sp = _made(prob_sum, "prob_sum", (experts,), torch.float32, device, dev)
        loss, op = _made(loss, "loss", (1,), torch.float32, device, dev)
        wsp, need, workspace = _workspace(workspace, _router_bytes(tokens, experts), device, dev)
        out += (counts, prob_sum, loss)
    bp = _maybe(bias, "bias", (experts,), _F32, dev)
    mp = _maybe(mask, "mask", (tokens,), _MASK, dev)
    _run(_library.situ_moe_router, handle, _ROUTER,
         tokens, experts, top_k, scoring, _out_code(logits.dtype), code, renormalize, scale, stride, lp, bp, mp, ip,
         wp, pp, cp, sp, op, wsp, need)
    return out


def situ_moe_router_backward(logits, ids, d_weights=None, *, scoring="softmax", renormalize=True, scale=1.0, mask=None,
                             counts=None, d_loss=None, out=None, out_dtype=None, stream=None):
    """The logits' gradient [tokens, experts] (in their type, or out_dtype) of
    situ_moe_router with the same arguments: through the weights from d_weights
    (fp32 [tokens, top_k]) and through the balance loss from counts (those of
    the loss) and d_loss (fp32 [1]); either may be None.  ids and counts are
    constants of it.  Rows of masked tokens are 0."""
    if torch is None:
        _first()
    dev, tokens, experts, stride, lp = _lead(logits, "logits", _EITHER)
    args = (logits, dev, tokens, experts, stride, lp, ids, d_weights, _scoring(scoring), bool(renormalize), scale,
            mask, counts, d_loss, out, out_dtype)
    if stream is None and dev == _device():
        return _router_backward(_raw_stream(dev), *args)
    return _elsewhere(dev, stream, _router_backward, *args)


def _router_backward(handle, logits, dev, tokens, experts, stride, lp, ids, d_weights, scoring, renormalize, scale,
                     mask,
                     counts, d_loss, out, out_dtype):
    if ids is None or ids.dim() != 2:          # the loss alone takes top_k from them
        _bad(ids, "ids", _INT32, dev, "[tokens, top_k]")
    top_k = ids.shape[1]
    ip = _dense(ids, "ids", (tokens, top_k), _INT32, dev)
    dp = _maybe(d_weights, "d_weights", (tokens, top_k), _F32, dev)
    mp = _maybe(mask, "mask", (tokens,), _MASK, dev)
    cp = _maybe(counts, "counts", (experts,), _INT32, dev)
    if d_loss is not None and d_loss.dim() == 0:
        d_loss = d_loss.view(1)
    gp = _maybe(d_loss, "d_loss", (1,), _F32, dev)
    if out is None:
        out = _empty(tokens, experts, dtype=out_dtype or logits.dtype, device=logits.device)
    elif out_dtype is not None and out.dtype != out_dtype:
        _bad(out, "out", (out_dtype,), dev, f"({tokens}, {experts})")
    code = _out_code(out.dtype)
    _, out_stride, op = _rows(out, "out", tokens, experts, _EITHER, dev)
    _run(_library.situ_moe_router_backward, handle, _ROUTER_BACKWARD,
         tokens, experts, top_k, scoring, _out_code(logits.dtype), code, renormalize, scale, stride, out_stride, lp,
         mp, ip, dp, cp, gp, op)
    return out


def _groups(activation, situ_beta, situ_linear_beta, swiglu_alpha, swiglu_beta, offsets, dev):
    """Code, experts and addresses of offsets and constants."""
    if offsets is None:
        experts, op = 1, 0
    else:
        experts = offsets.numel() - 1
        op = _dense(offsets, "offsets", (experts + 1,), _INT32, dev)
    if activation == "situ":
        return (0, experts, op, _dense(situ_beta, "situ_beta", (experts,), _F32, dev),
                _dense(situ_linear_beta, "situ_linear_beta", (experts,), _F32, dev))
    if activation == "swiglu":
        return 1, experts, op, 0, 0
    if activation == "swiglu_bias":
        return (2, experts, op, _dense(swiglu_alpha, "swiglu_alpha", (experts,), _F32, dev),
                _dense(swiglu_beta, "swiglu_beta", (experts,), _F32, dev))
    _fail(3, f"activation {activation!r} ({', '.join(_B.ACTIVATIONS)})")


def situ_moe_activation(gate_up, *, activation="situ", situ_beta=None, situ_linear_beta=None, swiglu_alpha=None,
                        swiglu_beta=None, offsets=None, out=None, checkpoint=False, codes=None, scales=None, stream=None):
    """h = act(gate, up), bf16 [rows, I], of gate_up bf16 [rows, 2I] (gate
    columns first; a row stride is allowed), the rows grouped by expert through
    offsets int32 [experts + 1] (None: one group).  I a multiple of 8.

    activation: situ (situ_beta, situ_linear_beta fp32 [experts]), swiglu, or
    swiglu_bias (swiglu_alpha, swiglu_beta).  checkpoint=True (or codes and
    scales given) also keeps gate_up in 8 bits for
    situ_moe_activation_backward: E4M3 codes uint8 [rows, 2I] and fp32 scales
    [rows, 2 ceil(I / 128)], and returns (h, codes, scales).  Rows outside
    every group are left as they are (undefined in an output allocated here)."""
    if torch is None:
        _first()
    dev, rows, width, stride, gp = _lead(gate_up, "gate_up", _BF16)
    args = (gate_up.device, dev, rows, width, stride, gp, activation, situ_beta, situ_linear_beta, swiglu_alpha,
            swiglu_beta, offsets, out, checkpoint, codes, scales)
    if stream is None and dev == _device():
        return _activation(_raw_stream(dev), *args)
    return _elsewhere(dev, stream, _activation, *args)


def _activation(handle, device, dev, rows, width, stride, gp, activation, situ_beta, situ_linear_beta, swiglu_alpha,
                swiglu_beta, offsets, out, checkpoint, codes, scales):
    if width % 16:
        _fail(2, f"gate_up has {width} columns, not a multiple of 16")
    inner = width // 2
    code, experts, op, p0, p1 = _groups(activation, situ_beta, situ_linear_beta, swiglu_alpha, swiglu_beta, offsets, dev)
    if out is None:
        out = _empty(rows, inner, dtype=torch.bfloat16, device=device)
        h_stride, hp = inner, out.data_ptr()
    else:
        _, h_stride, hp = _rows(out, "out", rows, inner, _BF16, dev)
    cp = sp = 0
    if checkpoint or codes is not None or scales is not None:
        checkpoint = True
        shape = (rows, 2 * -(-inner // 128))
        if codes is None:
            codes = _empty(rows, width, dtype=torch.uint8, device=device)
            cp = codes.data_ptr()
        else:
            cp = _dense(codes, "codes", (rows, width), _CODES, dev)
        scales, sp = _made(scales, "scales", shape, torch.float32, device, dev)
    _run(_library.situ_moe_activation, handle, _ACTIVATION,
         rows, inner, experts, code, stride, h_stride, 0, 0, op, p0, p1, gp, hp, cp, sp, 0, 0)
    return (out, codes, scales) if checkpoint else out


def situ_moe_activation_backward(dh, gate_up, scales=None, *, activation="situ", situ_beta=None, situ_linear_beta=None,
                                 swiglu_alpha=None, swiglu_beta=None, offsets=None, out=None, recompute=False, h=None,
                                 stream=None):
    """The gradient of situ_moe_activation in gate_up, bf16 [rows, 2I], from dh
    bf16 [rows, I] and gate_up: the bf16 rows themselves, or with scales the
    codes that were kept.  recompute=True (or h given) also returns h at those
    values, (d_gate_up, h): the down product's input for its wgrad.  The
    activation's constants get no gradient."""
    if torch is None:
        _first()
    dev, rows, inner, stride, dp = _lead(dh, "dh", _BF16)
    args = (dh.device, dev, rows, inner, stride, dp, gate_up, scales, activation, situ_beta, situ_linear_beta,
            swiglu_alpha, swiglu_beta, offsets, out, recompute, h)
    if stream is None and dev == _device():
        return _activation_backward(_raw_stream(dev), *args)
    return _elsewhere(dev, stream, _activation_backward, *args)


def _activation_backward(handle, device, dev, rows, inner, stride, dp, gate_up, scales, activation, situ_beta,
                         situ_linear_beta, swiglu_alpha, swiglu_beta, offsets, out,
                         recompute, h):
    if inner % 8:
        _fail(2, f"dh has {inner} columns, not a multiple of 8")
    code, experts, op, p0, p1 = _groups(activation, situ_beta, situ_linear_beta, swiglu_alpha, swiglu_beta, offsets, dev)
    g_stride = gp = cp = sp = 0
    if scales is None:
        _, g_stride, gp = _rows(gate_up, "gate_up", rows, 2 * inner, _BF16, dev)
    else:
        cp = _dense(gate_up, "gate_up", (rows, 2 * inner), _CODES, dev)
        sp = _dense(scales, "scales", (rows, 2 * -(-inner // 128)), _F32, dev)
    if out is None:
        out = _empty(rows, 2 * inner, dtype=torch.bfloat16, device=device)
        o_stride, outp = 2 * inner, out.data_ptr()
    else:
        _, o_stride, outp = _rows(out, "out", rows, 2 * inner, _BF16, dev)
    h_stride = hp = 0
    if h is not None:
        recompute = True
        _, h_stride, hp = _rows(h, "h", rows, inner, _BF16, dev)
    elif recompute:
        h = _empty(rows, inner, dtype=torch.bfloat16, device=device)
        h_stride, hp = inner, h.data_ptr()
    _run(_library.situ_moe_activation_backward, handle, _ACTIVATION,
         rows, inner, experts, code, g_stride, h_stride, stride, o_stride, op, p0, p1, gp, hp, cp, sp, dp, outp)
    return (out, h) if recompute else out


def _pairs(weights, inv, dev):
    """Tokens, slots and addresses of weights [tokens, top_k] and inv (of as many)."""
    if weights is None or weights.dim() != 2 or weights.dtype not in _EITHER:
        _bad(weights, "weights", _EITHER, dev, "[tokens, top_k]")
    tokens, top_k = weights.shape
    wp = _dense(weights, "weights", (tokens, top_k), _EITHER, dev)
    if inv is None or inv.dim() != 1:
        ip = _dense(inv, "inv", (tokens, top_k), _INT32, dev)
    else:
        ip = _dense(inv, "inv", (tokens * top_k,), _INT32, dev)
    return tokens, top_k, wp, ip


def situ_moe_combine(y, weights, inv, *, out=None, out_dtype=None, stream=None):
    """out[t] = sum over slots s of weights[t, s] y[inv[t, s]], [tokens,
    hidden] in bf16 (the default) or fp32, summed in fp32 in slot order.

    y: bf16 or fp32 [rows, hidden] (hidden a multiple of 8); weights: bf16 or
    fp32 [tokens, top_k]; inv: int32 [tokens, top_k] or [tokens * top_k], the
    row of each pair as situ_moe_route leaves it (outside [0, rows): the pair
    is not local)."""
    if torch is None:
        _first()
    dev, rows, hidden, stride, yp = _lead(y, "y", _EITHER)
    args = (y, dev, rows, hidden, stride, yp, weights, inv, out, out_dtype)
    if stream is None and dev == _device():
        return _combine(_raw_stream(dev), *args)
    return _elsewhere(dev, stream, _combine, *args)


def _combine(handle, y, dev, rows, hidden, stride, yp, weights, inv, out, out_dtype):
    tokens, top_k, wp, ip = _pairs(weights, inv, dev)
    if out is None:
        out = _empty(tokens, hidden, dtype=out_dtype or torch.bfloat16, device=y.device)
    elif out_dtype is not None and out.dtype != out_dtype:
        _bad(out, "out", (out_dtype,), dev, f"({tokens}, {hidden})")
    code = _out_code(out.dtype)
    _, out_stride, op = _rows(out, "out", tokens, hidden, _EITHER, dev)
    _run(_library.situ_moe_combine, handle, _COMBINE,
         tokens, top_k, hidden, rows, _out_code(y.dtype), _out_code(weights.dtype), code, 0, stride, out_stride, 0,
         yp, wp, ip, op, 0, 0)
    return out


def situ_moe_combine_backward(d_out, y, weights, inv, *, dy=None, d_weights=None, stream=None):
    """The gradients of situ_moe_combine: dy[inv[t, s]] = weights[t, s]
    d_out[t], in y's type, and d_weights[t, s] = d_out[t] . y[inv[t, s]] in
    fp32 (0 where the pair is not local).  d_out: bf16 or fp32 [tokens,
    hidden].  Each row of y belongs to one pair at most; rows of no pair are
    left as they are (undefined in a dy allocated here).  Returns (dy,
    d_weights)."""
    if torch is None:
        _first()
    dev, rows, hidden, stride, yp = _lead(y, "y", _EITHER)
    args = (d_out, y, dev, rows, hidden, stride, yp, weights, inv, dy, d_weights)
    if stream is None and dev == _device():
        return _combine_backward(_raw_stream(dev), *args)
    return _elsewhere(dev, stream, _combine_backward, *args)


def _combine_backward(handle, d_out, y, dev, rows, hidden, stride, yp, weights, inv, dy, d_weights):
    tokens, top_k, wp, ip = _pairs(weights, inv, dev)
    _, d_stride, dp = _rows(d_out, "d_out", tokens, hidden, _EITHER, dev)
    if dy is None:
        dy = _empty(rows, hidden, dtype=y.dtype, device=y.device)
        dy_stride, dyp = hidden, dy.data_ptr()
    else:
        _, dy_stride, dyp = _rows(dy, "dy", rows, hidden, (y.dtype,), dev)
    d_weights, gp = _made(d_weights, "d_weights", (tokens, top_k), torch.float32, y.device, dev)
    _run(_library.situ_moe_combine_backward, handle, _COMBINE,
         tokens, top_k, hidden, rows, _out_code(y.dtype), _out_code(weights.dtype), _out_code(d_out.dtype), 0, stride,
         d_stride, dy_stride, yp, wp, ip, dp, dyp, gp)
    return dy, d_weights


def situ_moe_adapters(x, a, b, offsets, adapter, *, base=None, ranks=None, scales=None, out=None, out_dtype=None,
                      workspace=None, stream=None):
    """out[r] = base[r] + scales[i] * b[i] (a[i] x[r]) for the rows r =
    offsets[q] .. offsets[q + 1] - 1 of each request q, i = adapter[q]; a
    request whose adapter is outside [0, adapters) has none, and its rows are
    base's.

    x: bf16 [rows, k]; a: bf16 [adapters, rank, k]; b: bf16 [adapters, n,
    rank]; offsets: int32 [requests + 1]; adapter: int32 [requests]; base: bf16
    or fp32 [rows, n], the shared projection's output (None: zeros); ranks:
    int32 [adapters], how many of a's rows count (None: all); scales: fp32
    [adapters] (None: 1).  k, n and rank multiples of 8, rank up to 256.  out:
    [rows, n] of base's type, or out_dtype (bf16) without one; it may be base
    itself.  Rows of no request are left as they are (undefined in an output
    allocated here)."""
    if torch is None:
        _first()
    dev, rows, k, stride, xp = _lead(x, "x", _BF16)
    args = (x.device, dev, rows, k, stride, xp, a, b, offsets, adapter, base, ranks, scales, out, out_dtype, workspace)
    if stream is None and dev == _device():
        return _adapters(_raw_stream(dev), *args)
    return _elsewhere(dev, stream, _adapters, *args)


def _adapters(handle, device, dev, rows, k, stride, xp, a, b, offsets, adapter, base, ranks, scales, out, out_dtype,
              workspace):
    if a is None or a.dim() != 3:
        _bad(a, "a", _BF16, dev, "[adapters, rank, k]")
    if b is None or b.dim() != 3:
        _bad(b, "b", _BF16, dev, "[adapters, n, rank]")
    held, rank, _ = a.shape
    n = b.shape[1]
    ap = _dense(a, "a", (held, rank, k), _BF16, dev)
    bp = _dense(b, "b", (held, n, rank), _BF16, dev)
    if offsets is None:
        _fail(1, "offsets is None")
    requests = offsets.numel() - 1
    op = _dense(offsets, "offsets", (requests + 1,), _INT32, dev)
    ip = _dense(adapter, "adapter", (requests,), _INT32, dev)
    rp = _maybe(ranks, "ranks", (held,), _INT32, dev)
    sp = _maybe(scales, "scales", (held,), _F32, dev)
    if out is None:
        dtype = out_dtype or (torch.bfloat16 if base is None else base.dtype)
        out = _empty(rows, n, dtype=dtype, device=device)
        code, o_stride, outp = _out_code(dtype), n, out.data_ptr()
    else:
        if out_dtype is not None and out.dtype != out_dtype:
            _bad(out, "out", (out_dtype,), dev, f"({rows}, {n})")
        code = _out_code(out.dtype)
        _, o_stride, outp = _rows(out, "out", rows, n, _EITHER, dev)
    b_stride = basep = 0
    if base is not None:
        _, b_stride, basep = _rows(base, "base", rows, n, (out.dtype,), dev)
    wsp, need, workspace = _workspace(workspace, _adapters_bytes(rows, n, k, rank, requests), device, dev)
    _run(_library.situ_moe_adapters, handle, _ADAPTERS,
         rows, n, k, rank, requests, held, code, 0, stride, b_stride, o_stride, op, ip, rp, sp, xp, ap, bp, basep,
         outp, wsp, need)
    return out
