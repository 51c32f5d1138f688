"""Cases of the 8-bit block-scaled products and the products grouped by expert.

A case names one pass through one operator:

  quantize  bf16 rows to E4M3 with one fp32 scale per row and 128 columns
  dense     out = (a * a_scale) (w * w_scale)^T, E4M3 with scales per 128
            (a: per row and 128 columns; w: per 128 x 128 block)
  experts   the same product with the rows grouped by expert, ragged
  forward   bf16 rows grouped by expert, out[r] = x[r] w_e^T
  backward  its gradients: dx[r] = dy[r] w_e and dw_e = sum_r dy[r]^T x[r]

`run` takes the elementary torch form of each in 32 bits, or, where `own` is
true, the calls a user makes of block_scaled_mxfp4_amd.
"""

import numpy as np
import torch

own = False

F8 = torch.float8_e4m3fn
F8_MAX = 448.0
TINY = 2.0 ** -100          # the smallest block maximum a scale is made from
OUT = {"bf16": torch.bfloat16, "f32": torch.float32}


def blocks(n):
    return -(-n // 128)


# ------------------------------------------------------------------ cases

def listed():
    return [
        # the activations of a small decode batch
        {"name": "quantize_decode", "op": "quantize", "rows": 64, "cols": 3584, "pad": 0},
        # the activations of a prefill batch
        {"name": "quantize_prefill", "op": "quantize", "rows": 32768, "cols": 3584, "pad": 0},
        # a dense projection beside the experts, one token
        {"name": "dense_one_token", "op": "dense", "rows": 1, "n": 3584, "k": 3584, "pad": 0, "out": "bf16"},
        # an odd decode batch, weight rows that end inside a scale block
        {"name": "dense_decode", "op": "dense", "rows": 45, "n": 2000, "k": 7168, "pad": 0, "out": "bf16"},
        # a prefill batch through a dense projection
        {"name": "dense_prefill", "op": "dense", "rows": 8192, "n": 7168, "k": 3584, "pad": 0, "out": "bf16"},
        # decode on an EP8 shard whose experts' gate and up rows are split over TP8
        {"name": "experts_decode", "op": "experts", "rows": 256, "experts": 112, "active": 100, "n": 768, "k": 3584,
         "pad": 0, "out": "f32"},
        # prefill on an EP8 shard, gate and up rows split over TP4
        {"name": "experts_prefill", "op": "experts", "rows": 16384, "experts": 112, "active": 104, "n": 1536,
         "k": 3584, "pad": 0, "out": "bf16"},
        # the down product of a gate_up adapter at decode: a token's row read for each of its local pairs
        {"name": "adapter_decode", "op": "forward", "rows": 128, "experts": 112, "active": 76, "n": 16, "k": 3584,
         "tokens": 64, "top_k": 16, "gather": True, "scatter": False, "out": "bf16"},
        # its up product at prefill, written to the rows of gate_up_lora_delta
        {"name": "adapter_prefill", "op": "forward", "rows": 16384, "experts": 112, "active": 104, "n": 768, "k": 32,
         "tokens": 8192, "top_k": 16, "gather": False, "scatter": True, "out": "bf16"},
        # bf16 expert weights at prefill
        {"name": "forward_prefill", "op": "forward", "rows": 16384, "experts": 16, "active": 16, "n": 1536, "k": 3584,
         "tokens": 0, "top_k": 1, "gather": False, "scatter": False, "out": "bf16"},
        # a training step's gradients of an adapter's down product
        {"name": "adapter_training", "op": "backward", "rows": 8192, "experts": 112, "active": 104, "n": 32,
         "k": 3584, "tokens": 4096, "top_k": 16, "gather": True, "out": "bf16"},
        # a training step's gradients of bf16 expert weights, an odd number of rows
        {"name": "backward_training", "op": "backward", "rows": 8191, "experts": 16, "active": 15, "n": 1536,
         "k": 3584, "tokens": 0, "top_k": 1, "gather": False, "out": "bf16"},
    ]


def draw(rng):
    def spread(lo, hi, step=1):
        """A multiple of `step`, its logarithm spread evenly over [lo, hi]."""
        v = int(round(lo * (hi / lo) ** rng.random() / step)) * step
        return min(max(v, -(-lo // step) * step), hi // step * step)

    op = rng.choice(["quantize", "dense", "experts", "forward", "backward"])
    if op == "quantize":
        cols = spread(16, 16384, 16)
        return {"op": op, "rows": spread(1, max(1, min(65536, (1 << 27) // cols))), "cols": cols,
                "pad": rng.choice([0, 0, 16, 256])}
    if op == "dense":
        n, k = spread(16, 8192), spread(64, 8192, 16)
        return {"op": op, "rows": spread(1, max(1, min(16384, (1 << 37) // (n * k)))), "n": n, "k": k,
                "pad": rng.choice([0, 0, 16, 128]), "out": rng.choice(["bf16", "f32"])}
    experts = spread(1, 128)
    if op == "experts":
        n, k = spread(16, 2048), spread(64, 4096, 16)
        rows = spread(1, max(1, min(16384, (1 << 36) // (n * k))))
        most = min(rows, experts)
        return {"op": op, "rows": rows, "experts": experts, "active": rng.randint(-(-most // 2), most), "n": n, "k": k,
                "pad": rng.choice([0, 0, 16, 128]), "out": rng.choice(["bf16", "f32"])}
    # adapters' ranks on one side, or whole expert matrices
    n, k = rng.choice([(spread(8, 64, 8), spread(64, 4096, 8)), (spread(64, 2048, 8), spread(8, 64, 8)),
                       (spread(64, 2048, 8), spread(64, 4096, 8))])
    rows = spread(1, max(1, min(16384, (1 << 36) // (n * k))))
    top_k = rng.randint(1, 16)
    experts = min(experts, (1 << 27) // (n * k))
    most = min(rows, experts)
    case = {"op": op, "rows": rows, "experts": experts, "active": rng.randint(-(-most // 2), most), "n": n, "k": k,
            "tokens": -(-rows * rng.randint(1, 8) // top_k), "top_k": top_k, "gather": rng.random() < 0.5,
            "out": rng.choice(["bf16", "f32"])}
    if op == "forward":
        case["scatter"] = rng.random() < 0.5
    return case


# ----------------------------------------------------------------- inputs

def _offsets(case, np_rng):
    """Rows per expert: `active` experts share the rows unevenly, each with one at least; the first row of each."""
    e, a, r = case["experts"], case["active"], case["rows"]
    share = np_rng.lognormal(0.0, 0.5, a)
    counts = np.zeros(e, np.int64)
    counts[np_rng.permutation(e)[:a]] = 1 + np_rng.multinomial(r - a, share / share.sum())
    return np.concatenate([[0], np.cumsum(counts)]).astype(np.int32), int(counts.max())


def _rows8(gen, rows, cols, pad):
    """E4M3 rows of normal values with a scale per 128 columns, as quantized activations are; the row stride has
    `pad` bytes more."""
    x = torch.randn(rows, blocks(cols), 128, generator=gen, device="cuda")
    scale = x.abs().amax(2) / F8_MAX
    codes = (x / scale[..., None]).to(F8).view(torch.uint8).reshape(rows, -1)[:, :cols]
    whole = torch.empty(rows, cols + pad, dtype=torch.uint8, device="cuda")
    whole[:, :cols] = codes
    return whole[:, :cols], scale


def _weights8(gen, e, n, k):
    """E4M3 expert weights of about unit gain with a scale for each block of 128 x 128."""
    codes = torch.empty(e, n, k, dtype=torch.uint8, device="cuda")
    for i in range(e):   # expert by expert: the wide values of all of them need not be held at once
        codes[i] = (torch.randn(n, k, generator=gen, device="cuda") * 100.0).clamp(-F8_MAX, F8_MAX).to(F8).view(torch.uint8)
    scale = (0.5 + torch.rand(e, blocks(n), blocks(k), generator=gen, device="cuda")) * (0.01 / k ** 0.5)
    return codes, scale


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    np_rng = np.random.RandomState(int(seed) % (1 << 31))
    s = dict(case)
    op = case["op"]
    if op == "quantize":
        whole = torch.randn(case["rows"], case["cols"] + case["pad"], generator=gen, device="cuda")
        s["x"] = (whole * torch.exp(torch.randn(case["rows"], 1, generator=gen, device="cuda"))).to(torch.bfloat16)[:, :case["cols"]]
        return s
    if op in ("dense", "experts"):
        s["a"], s["a_scale"] = _rows8(gen, case["rows"], case["k"], case["pad"])
        e = case["experts"] if op == "experts" else 1
        s["w"], s["w_scale"] = _weights8(gen, e, case["n"], case["k"])
        if op == "dense":
            s["w"], s["w_scale"] = s["w"][0], s["w_scale"][0]
            return s
    offsets, s["most"] = _offsets(case, np_rng)
    s["offsets"] = torch.from_numpy(offsets).cuda()
    if op == "experts":
        return s
    rows, n, k, e = case["rows"], case["n"], case["k"], case["experts"]
    s["w"] = (torch.randn(e, n, k, generator=gen, device="cuda") / k ** 0.5).to(torch.bfloat16)
    s["pairs"] = None
    s["x_div"] = s["out_div"] = 0
    x_rows = rows
    if case["gather"] or case.get("scatter"):
        # position r stands for pair pairs[r] = token * top_k + slot, ascending within an expert
        pick = np_rng.permutation(case["tokens"] * case["top_k"])[:rows]
        order = np.lexsort((pick, np.repeat(np.arange(e), np.diff(offsets))))
        s["pairs"] = torch.from_numpy(pick[order].astype(np.int32)).cuda()
        if case["gather"]:
            s["x_div"], x_rows = case["top_k"], case["tokens"]
        if case.get("scatter"):
            s["out_div"] = 1
            s["held"] = torch.zeros(case["tokens"] * case["top_k"], n, dtype=OUT[case["out"]], device="cuda")
    s["x"] = torch.randn(x_rows, k, generator=gen, device="cuda").to(torch.bfloat16)
    if op == "backward":
        s["dy"] = torch.randn(rows, n, generator=gen, device="cuda").to(torch.bfloat16)
    return s


# ------------------------------------------------------------ plain forms

def _quantize(x):
    rows, cols = x.shape
    f = torch.nn.functional.pad(x.float(), (0, 128 * blocks(cols) - cols)).view(rows, -1, 128)
    scale = f.abs().amax(2).clamp(min=TINY) / F8_MAX
    return (f / scale[..., None]).to(F8).view(rows, -1)[:, :cols], scale


def _wide(codes, scale, block_rows):
    """E4M3 codes times their scales in 32 bits."""
    n, k = codes.shape[-2:]
    full = scale.repeat_interleave(128, -1)[..., :k]
    if block_rows:
        full = full.repeat_interleave(128, -2)[..., :n, :]
    return codes.contiguous().view(F8).float() * full


def _padded(s):
    """[experts, most] row of each place of each expert, and which places hold one."""
    first, last = s["offsets"][:-1, None].long(), s["offsets"][1:, None].long()
    at = first + torch.arange(s["most"], device="cuda")
    held = at < last
    return torch.where(held, at, 0), held


def _unpadded(s, y):
    """The rows in their order again, from [experts, most, ...]."""
    r = torch.arange(s["rows"], device="cuda")
    e = torch.searchsorted(s["offsets"][1:].long(), r, right=True)
    return y[e, r - s["offsets"].long()[e]]


def _x_rows(s, at):
    return s["pairs"].long()[at] // s["x_div"] if s["x_div"] else at


def _plain(s):
    op = s["op"]
    if op == "quantize":
        return _quantize(s["x"])
    out = OUT[s["out"]]
    if op == "dense":
        return (_wide(s["a"], s["a_scale"], False) @ _wide(s["w"], s["w_scale"], True).t()).to(out)
    at, held = _padded(s)
    if op == "experts":
        a = _wide(s["a"], s["a_scale"], False)[at] * held[..., None]
        return _unpadded(s, torch.bmm(a, _wide(s["w"], s["w_scale"], True).transpose(1, 2))).to(out)
    x = s["x"].float()[_x_rows(s, at)] * held[..., None]
    if op == "forward":
        y = _unpadded(s, torch.bmm(x, s["w"].float().transpose(1, 2))).to(out)
        if s["out_div"]:
            s["held"][s["pairs"].long()] = y
            return s["held"]
        return y
    dy = s["dy"].float()[at] * held[..., None]
    return {"dx": _unpadded(s, torch.bmm(dy, s["w"].float())).to(out), "dw": torch.bmm(dy.transpose(1, 2), x)}


# --------------------------------------------------------- the framework's

def _calls(s):
    import block_scaled_mxfp4_amd as B
    op = s["op"]
    if op == "quantize":
        codes, scales = B.situ_moe_quantize_fp8_block128(s["x"])
        return codes.view(F8), scales
    out = OUT[s["out"]]
    if op in ("dense", "experts"):
        return B.situ_moe_matmul_fp8_block128(s["a"], s["a_scale"], s["w"], s["w_scale"], offsets=s.get("offsets"),
                                              out_dtype=out)
    if op == "forward":
        return B.situ_moe_grouped_matmul(s["x"], s["w"], s["offsets"], pairs=s["pairs"], x_div=s["x_div"],
                                         out_div=s["out_div"], out=s.get("held"), out_dtype=out)
    return {"dx": B.situ_moe_grouped_matmul_dgrad(s["dy"], s["w"], s["offsets"], out_dtype=out),
            "dw": B.situ_moe_grouped_matmul_wgrad(s["dy"], s["x"], s["offsets"], pairs=s["pairs"], x_div=s["x_div"],
                                                  out_dtype=torch.float32)}


def run(state):
    return _calls(state) if own else _plain(state)


# ------------------------------------------------------- work and 64 bits

def work(case):
    op = case["op"]
    if op == "quantize":
        n = case["rows"] * case["cols"]
        return {"bytes": 3 * n + 4 * case["rows"] * blocks(case["cols"]), "flops": 2 * n}
    rows, n, k = case["rows"], case["n"], case["k"]
    size = 2 if case["out"] == "bf16" else 4
    flops = 2 * rows * n * k
    if op in ("dense", "experts"):
        e = case.get("active", 1)
        return {"bytes": rows * (k + 4 * blocks(k)) + e * (n * k + 4 * blocks(n) * blocks(k)) + size * rows * n,
                "flops": flops}
    x_rows = min(rows, case["tokens"]) if case["gather"] else rows
    if op == "forward":
        return {"bytes": 2 * x_rows * k + 2 * case["active"] * n * k + size * rows * n, "flops": flops}
    return {"bytes": 2 * rows * n + 2 * x_rows * k + 2 * case["active"] * n * k + size * rows * k
            + 4 * case["experts"] * n * k, "flops": 2 * flops}


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    d = torch.float64
    if op == "quantize":
        x, scales, codes = s["x"].to(d), [], []
        for c in range(0, case["cols"], 128):
            part = x[:, c:c + 128]
            scales.append(torch.clamp(part.abs().max(dim=1).values, min=TINY) / F8_MAX)
            codes.append(part / scales[-1][:, None])
        return torch.cat(codes, 1), torch.stack(scales, 1)
    rows, n, k = case["rows"], case["n"], case["k"]
    if op in ("dense", "experts"):
        bounds = [0, rows] if op == "dense" else s["offsets"].tolist()
        w, ws = s["w"].view(-1, n, k), s["w_scale"].view(-1, blocks(n), blocks(k))
        out = torch.zeros(rows, n, dtype=d, device="cuda")
        columns, lines = torch.arange(k, device="cuda") // 128, torch.arange(n, device="cuda") // 128
        for e, (lo, hi) in enumerate(zip(bounds[:-1], bounds[1:])):
            if hi > lo:
                a = s["a"][lo:hi].contiguous().view(F8).to(d) * s["a_scale"][lo:hi].to(d)[:, columns]
                out[lo:hi] = a @ (w[e].view(F8).to(d) * ws[e].to(d)[lines][:, columns]).t()
        return out
    bounds = s["offsets"].tolist()
    pairs = s["pairs"].long() if s["pairs"] is not None else None
    x = s["x"][pairs // s["x_div"]] if s["x_div"] else s["x"]
    if op == "forward":
        out = torch.zeros(rows, n, dtype=d, device="cuda")
        for e, (lo, hi) in enumerate(zip(bounds[:-1], bounds[1:])):
            if hi > lo:
                out[lo:hi] = x[lo:hi].to(d) @ s["w"][e].to(d).t()
        if s["out_div"]:
            whole = torch.zeros(s["held"].shape, dtype=d, device="cuda")
            whole[pairs] = out
            return whole
        return out
    dx = torch.zeros(rows, k, dtype=d, device="cuda")
    dw = torch.zeros(case["experts"], n, k, dtype=d, device="cuda")
    for e, (lo, hi) in enumerate(zip(bounds[:-1], bounds[1:])):
        if hi > lo:
            dy = s["dy"][lo:hi].to(d)
            dx[lo:hi] = dy @ s["w"][e].to(d)
            dw[e] = dy.t() @ x[lo:hi].to(d)
    return {"dx": dx, "dw": dw}
