"""Cases of the operators around the routed products: the gate in front of them,
the gated activation between them, the combine behind them, with their
gradients, and low-rank adapters of many requests beside a shared projection.

A case names one pass through one operator:

  router               expert ids and weights of each token from its logits; with
                       `balance` the tokens per expert and the balance loss too
  router_backward      the logits' gradient from the weights' and the loss's
  activation           h = act(gate, up); with `keep` gate and up are also kept in 8 bits
  activation_backward  gate's and up's gradient, and h again, from what was kept
  combine              the weighted sum of a token's expert rows
  combine_backward     the expert rows' and the weights' gradients
  adapters             base + c_a B_a (A_a x) for the rows of requests with an adapter each

`run` takes the elementary torch form of each in 32 bits, or, where `own` is
true, the calls a user makes of block_scaled_mxfp4_amd.
"""

import numpy as np
import torch

own = False

F8 = torch.float8_e4m3fn
F8_MAX = 448.0
TINY = 2.0 ** -100          # the smallest block maximum a scale is made from
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
NOTHING = float("-inf")


def blocks(n):
    return -(-n // 128)


# ------------------------------------------------------------------ cases

def listed():
    return [
        # serving: one token of a decode step is routed
        {"name": "router_one_token", "op": "router", "tokens": 1, "experts": 896, "top_k": 16, "type": "f32",
         "scoring": "sigmoid", "bias": True, "renormalize": True, "balance": False, "closed": 0, "padded": 0},
        # a prefill batch of a training step, with the balance loss
        {"name": "router_prefill", "op": "router", "tokens": 32768, "experts": 896, "top_k": 16, "type": "f32",
         "scoring": "softmax", "bias": False, "renormalize": True, "balance": True, "closed": 0, "padded": 0},
        # a padded batch of an odd number of tokens, scores with a selection bias, bf16 logits
        {"name": "router_padded", "op": "router", "tokens": 8191, "experts": 112, "top_k": 8, "type": "bf16",
         "scoring": "sigmoid", "bias": True, "renormalize": True, "balance": True, "closed": 0, "padded": 700},
        # the way back of a training step through the gate
        {"name": "router_backward", "op": "router_backward", "tokens": 16384, "experts": 896, "top_k": 16,
         "type": "f32", "scoring": "softmax", "bias": False, "renormalize": True, "balance": True, "closed": 0,
         "padded": 0},
        # serving: a decode batch's pairs on a TP8 shard
        {"name": "activation_decode", "op": "activation", "rows": 1024, "inner": 384, "experts": 112, "active": 90,
         "kind": "situ", "keep": False},
        # a training step's pairs on a TP8 shard, gate and up kept in 8 bits
        {"name": "activation_kept", "op": "activation", "rows": 262144, "inner": 384, "experts": 896, "active": 896,
         "kind": "situ", "keep": True},
        # the way back of a few rows of ragged width
        {"name": "activation_backward_ragged", "op": "activation_backward", "rows": 1001, "inner": 200, "experts": 16,
         "active": 15, "kind": "swiglu", "keep": True},
        # the way back of a training step
        {"name": "activation_backward", "op": "activation_backward", "rows": 65521, "inner": 768, "experts": 112,
         "active": 104, "kind": "situ", "keep": True},
        # an EP8 shard's partial output: an eighth of the pairs are local
        {"name": "combine_shard", "op": "combine", "tokens": 8192, "top_k": 16, "local": 0.125, "hidden": 3584,
         "type": "bf16"},
        # the way back of a training step whose pairs are all local
        {"name": "combine_backward", "op": "combine_backward", "tokens": 4095, "top_k": 16, "local": 1.0,
         "hidden": 3584, "type": "bf16"},
        # serving: one token each of 64 requests, half as many adapters, some requests without
        {"name": "adapters_decode", "op": "adapters", "rows": 64, "requests": 64, "adapters": 32, "rank": 16,
         "k": 3584, "n": 7168, "type": "bf16"},
        # serving: a prefill batch of requests of uneven lengths
        {"name": "adapters_prefill", "op": "adapters", "rows": 8192, "requests": 13, "adapters": 8, "rank": 32,
         "k": 3584, "n": 7168, "type": "bf16"},
    ]


def draw(rng):
    def spread(lo, hi, step=1):
        """A multiple of `step`, its logarithm spread evenly over [lo, hi]."""
        v = int(round(lo * (hi / lo) ** rng.random() / step)) * step
        return min(max(v, -(-lo // step) * step), hi // step * step)

    op = rng.choice(["router", "router", "router_backward", "activation", "activation_backward", "combine",
                     "combine_backward", "adapters", "adapters"])
    if op.startswith("router"):
        experts = spread(8, 1024)
        tokens = spread(1, min(32768, (1 << 24) // experts))
        scoring = rng.choice(["softmax", "sigmoid"])
        return {"op": op, "tokens": tokens, "experts": experts, "top_k": spread(1, min(experts - experts // 8, 24)),
                "type": rng.choice(["f32", "bf16"]), "scoring": scoring,
                "bias": scoring == "sigmoid" and rng.random() < 0.5, "renormalize": rng.random() < 0.75,
                "balance": rng.random() < 0.5 or op == "router_backward",
                "closed": rng.choice([0, 0, experts // 8]), "padded": rng.choice([0, 0, tokens // 3])}
    if op.startswith("activation"):
        inner = spread(8, 4096, 8)
        rows = spread(1, min(131072, (1 << 26) // inner))
        experts = spread(1, 512)
        most = min(rows, experts)
        return {"op": op, "rows": rows, "inner": inner, "experts": experts, "active": rng.randint(-(-most // 2), most),
                "kind": rng.choice(["situ", "situ", "swiglu", "swiglu_bias"]), "keep": rng.random() < 0.6}
    if op.startswith("combine"):
        hidden, top_k = spread(64, 8192, 8), rng.randint(1, 16)
        return {"op": op, "tokens": spread(1, min(16384, (1 << 27) // (hidden * top_k))), "top_k": top_k,
                "local": rng.choice([1.0, 0.5, 0.125]), "hidden": hidden, "type": rng.choice(["bf16", "bf16", "f32"])}
    n, k = spread(64, 8192, 8), spread(64, 8192, 8)
    rows = spread(1, min(8192, (1 << 25) // max(n, k)))
    return {"op": op, "rows": rows, "requests": spread(1, min(rows, 256)), "adapters": spread(1, 48),
            "rank": rng.choice([8, 16, 16, 32, 64]), "k": k, "n": n, "type": rng.choice(["bf16", "bf16", "f32"])}


# ----------------------------------------------------------------- inputs

def _offsets(np_rng, rows, groups, active):
    """`active` of the groups share the rows unevenly, each with one at least; the first row of each."""
    share = np_rng.lognormal(0.0, 0.7, active)
    counts = np.zeros(groups, np.int64)
    counts[np_rng.permutation(groups)[:active]] = 1 + np_rng.multinomial(rows - active, share / share.sum())
    return np.concatenate([[0], np.cumsum(counts)]).astype(np.int32), int(counts.max())


def _logits(case, gen, np_rng, s):
    t, e = case["tokens"], case["experts"]
    favour = 0.5 * torch.randn(e, generator=gen, device="cuda")      # some experts are asked for more often
    z = torch.randn(t, e, generator=gen, device="cuda") + favour
    z[:, torch.from_numpy(np_rng.permutation(e)[:case["closed"]]).cuda()] = NOTHING
    s["logits"] = z.to(TYPES[case["type"]])
    s["bias"] = 0.1 * torch.randn(e, generator=gen, device="cuda") if case["bias"] else None
    s["mask"] = None
    if case["padded"]:
        s["mask"] = torch.arange(t, device="cuda") < t - case["padded"]
        s["logits"][t - case["padded"]:] = float("nan")


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    np_rng = np.random.RandomState(int(seed) % (1 << 31))
    s = dict(case)
    op = case["op"]

    def normal(*shape, scale=1.0, dtype=torch.bfloat16):
        return (scale * torch.randn(*shape, generator=gen, device="cuda")).to(dtype)

    if op.startswith("router"):
        _logits(case, gen, np_rng, s)
        s["scale"] = 2.5 if case["scoring"] == "sigmoid" else 1.0
        if op == "router_backward":
            s["ids"] = _choose(s)
            s["counts"] = _counts(s["ids"], case["experts"])
            s["d_weights"] = normal(case["tokens"], case["top_k"], dtype=torch.float32)
            s["d_loss"] = torch.full((1,), 0.01 * case["tokens"], device="cuda")
        return s
    if op.startswith("activation"):
        rows, inner, e = case["rows"], case["inner"], case["experts"]
        s["offsets"] = torch.from_numpy(_offsets(np_rng, rows, e, case["active"])[0]).cuda()
        width = torch.exp(0.5 * torch.randn(rows, 1, generator=gen, device="cuda"))
        s["gate_up"] = (torch.randn(rows, 2 * inner, generator=gen, device="cuda") * width).to(torch.bfloat16)
        # per expert: beta and linear beta, or alpha and beta
        s["p0"] = 0.5 + 1.5 * torch.rand(e, generator=gen, device="cuda")
        s["p1"] = 0.5 + 1.5 * torch.rand(e, generator=gen, device="cuda")
        if op == "activation_backward":
            s["d_out"] = normal(rows, inner)
            s["kept"] = (s["gate_up"], None)
            if case["keep"]:
                codes, scales = _keep(s["gate_up"], inner)
                s["kept"] = (codes.view(torch.uint8), scales)
            del s["gate_up"]
        return s
    if op.startswith("combine"):
        t, k, hidden = case["tokens"], case["top_k"], case["hidden"]
        pairs = t * k
        rows = max(1, round(case["local"] * pairs))
        inv = np.full(pairs, -1, np.int32)
        inv[np_rng.permutation(pairs)[:rows]] = np_rng.permutation(rows)
        s["inv"] = torch.from_numpy(inv).cuda().view(t, k)
        s["weights"] = torch.softmax(torch.randn(t, k, generator=gen, device="cuda"), 1).to(torch.bfloat16)
        s["y"] = normal(rows, hidden, dtype=TYPES[case["type"]])
        if op == "combine_backward":
            s["d_out"] = normal(t, hidden)
        return s
    rows, k, n, r, held = case["rows"], case["k"], case["n"], case["rank"], case["adapters"]
    offsets, s["most"] = _offsets(np_rng, rows, case["requests"], case["requests"])
    s["offsets"] = torch.from_numpy(offsets).cuda()
    s["ids"] = torch.from_numpy(np_rng.randint(-1, held, case["requests"]).astype(np.int32)).cuda()   # -1: none
    s["x"], s["base"] = normal(rows, k), normal(rows, n, dtype=TYPES[case["type"]])
    s["a"], s["b"] = normal(held, r, k, scale=k ** -0.5), normal(held, n, r, scale=r ** -0.5)
    s["scales"] = 0.5 + torch.rand(held, generator=gen, device="cuda")
    return s


# ------------------------------------------------------------ plain forms

def _choose(s):
    """Ids of the largest scores, the lowest first among equals; -1 where nothing is left to choose."""
    z = s["logits"].float()
    # sigmoid + bias in 64 bits: in 32 neighbours change places
    key = torch.sigmoid(s["logits"].double()) + s["bias"].double() if s["bias"] is not None else z
    key = torch.where(z > NOTHING, key, NOTHING)          # not NaN either
    if s["mask"] is not None:
        key = torch.where(s["mask"][:, None], key, NOTHING)
    top, ids = torch.sort(key, dim=1, descending=True, stable=True)
    ids = ids[:, :s["top_k"]]
    return torch.where(top[:, :s["top_k"]] > NOTHING, ids, -1).int()


def _counts(ids, experts):
    at = torch.where(ids < 0, experts, ids).long().flatten()
    return torch.zeros(experts + 1, dtype=torch.int32, device="cuda").index_add_(0, at, torch.ones_like(at, dtype=torch.int32))[:experts]


def _scores(s):
    """exp(z - max) or sigmoid(z), zero in masked rows."""
    z = s["logits"].float()
    if s["mask"] is not None:
        z = torch.where(s["mask"][:, None], z, 0.0)
    a = torch.exp(z - z.amax(1, keepdim=True)) if s["scoring"] == "softmax" else 1.0 / (1.0 + torch.exp(-z))
    return a if s["mask"] is None else a * s["mask"][:, None]


def _share(a):
    total = a.sum(1, keepdim=True)
    return a / torch.where(total > 0, total, 1.0)


def _router(s):
    a = _scores(s)
    ids = _choose(s)
    p = _share(a)
    chosen = torch.gather(p if s["scoring"] == "softmax" else a, 1, ids.long().clamp(min=0)) * (ids >= 0)
    weights = (s["scale"] * (_share(chosen) if s["renormalize"] else chosen)).to(torch.bfloat16)
    if not s["balance"]:
        return ids, weights
    counts, prob_sum = _counts(ids, s["experts"]), p.sum(0)
    c = counts.sum().float()
    loss = s["experts"] * s["top_k"] * (counts * prob_sum).sum() / torch.where(c > 0, c * c, 1.0)
    return ids, weights, counts, prob_sum, loss.view(1)


def _router_backward(s):
    a = _scores(s)
    p = _share(a)
    at, held = s["ids"].long().clamp(min=0), s["ids"] >= 0
    c = s["counts"].sum().float()
    g = s["d_loss"] * (s["experts"] * s["top_k"]) * s["counts"] / torch.where(c > 0, c * c, 1.0)
    dz = p * (g - (p * g).sum(1, keepdim=True))
    dw = s["d_weights"] * s["scale"] * held
    if s["renormalize"]:
        q = _share(torch.gather(a, 1, at) * held)
        dz = dz.scatter_add(1, at, q * (dw - (q * dw).sum(1, keepdim=True)))
        if s["scoring"] == "sigmoid":
            dz = dz * (1.0 - a)
    else:
        pick = torch.gather(p, 1, at) if s["scoring"] == "softmax" else torch.gather(a, 1, at)
        if s["scoring"] == "softmax":
            dz = dz.scatter_add(1, at, pick * dw) - p * (pick * dw).sum(1, keepdim=True)
        else:
            dz = (dz.scatter_add(1, at, pick * dw)) * (1.0 - a)
    if s["mask"] is not None:
        dz = torch.where(s["mask"][:, None], dz, 0.0)
    return dz.to(s["logits"].dtype)


def _keep(gate_up, inner):
    """Codes [rows, 2 inner] and scales [rows, 2 blocks] of the two halves."""
    rows, pad = gate_up.shape[0], 128 * blocks(inner) - inner
    f = torch.nn.functional.pad(gate_up.float().view(rows, 2, inner), (0, pad)).view(rows, 2, -1, 128)
    scale = f.abs().amax(3).clamp(min=TINY) / F8_MAX
    codes = (f / scale[..., None]).to(F8).view(rows, 2, -1)[..., :inner]
    return codes.reshape(rows, 2 * inner), scale.view(rows, -1)


def _halves(s):
    """Gate and up in 32 bits, as they were kept."""
    kept, scales = s["kept"]
    rows, inner = kept.shape[0], s["inner"]
    if scales is None:
        return kept[:, :inner].float(), kept[:, inner:].float()
    full = scales.view(rows, 2, -1).repeat_interleave(128, 2)[..., :inner]
    v = kept.view(F8).float().view(rows, 2, inner) * full
    return v[:, 0], v[:, 1]


def _per_row(s, p):
    """An expert's constant on each of its rows."""
    r = torch.arange(s["rows"], device="cuda")
    return p[torch.searchsorted(s["offsets"][1:].long(), r, right=True)][:, None]


def _gate(s, g):
    """The gate's factor and its derivative."""
    if s["kind"] == "situ":
        b = _per_row(s, s["p0"])
        t, o = torch.tanh(g / b), 1.0 / (1.0 + torch.exp(-g))
        # 1 - t^2 and 1 - o without cancellation
        left = torch.exp(-2.0 * (g / b).abs())
        slope = 4.0 * left / (1.0 + left) ** 2
        return b * t * o, slope * o + b * t * o / (1.0 + torch.exp(g))
    a = _per_row(s, s["p0"]) if s["kind"] == "swiglu_bias" else 1.0
    o = 1.0 / (1.0 + torch.exp(-a * g))
    return g * o, o + a * g * o / (1.0 + torch.exp(a * g))


def _up(s, u):
    if s["kind"] == "situ":
        b = _per_row(s, s["p1"])
        left = torch.exp(-2.0 * (u / b).abs())
        return b * torch.tanh(u / b), 4.0 * left / (1.0 + left) ** 2
    return (u + _per_row(s, s["p1"]) if s["kind"] == "swiglu_bias" else u), torch.ones_like(u)


def _activation(s):
    inner = s["inner"]
    g, u = s["gate_up"][:, :inner].float(), s["gate_up"][:, inner:].float()
    h = (_gate(s, g)[0] * _up(s, u)[0]).to(torch.bfloat16)
    return (h, *_keep(s["gate_up"], inner)) if s["keep"] else h


def _activation_backward(s):
    g, u = _halves(s)
    (a, da), (b, db) = _gate(s, g), _up(s, u)
    d = s["d_out"].float()
    return torch.cat([d * da * b, d * a * db], 1).to(torch.bfloat16), (a * b).to(torch.bfloat16)


def _pair_rows(s):
    local = s["inv"] >= 0
    return s["y"][s["inv"].long().clamp(min=0)].float() * local[..., None]


def _combine(s):
    return (s["weights"].float()[..., None] * _pair_rows(s)).sum(1).to(torch.bfloat16)


def _combine_backward(s):
    d = s["d_out"].float()
    dw = (_pair_rows(s) * d[:, None]).sum(2)
    at = torch.zeros(s["y"].shape[0] + 1, dtype=torch.long, device="cuda")     # the pair of each row
    pairs = torch.arange(s["inv"].numel(), device="cuda")
    at[s["inv"].flatten().long()] = pairs                                     # those that are not local: the last place
    at = at[:-1]
    dy = s["weights"].float().flatten()[at, None] * d[at // s["top_k"]]
    return dy.to(s["y"].dtype), dw


def _adapters(s):
    first, last = s["offsets"][:-1, None].long(), s["offsets"][1:, None].long()
    at = first + torch.arange(s["most"], device="cuda")
    held = at < last
    at = torch.where(held, at, 0)
    some = s["ids"] >= 0
    a = s["ids"].long().clamp(min=0)
    c = s["scales"][a] * some
    t = torch.bmm(s["x"].float()[at], s["a"].float()[a].transpose(1, 2)) * c[:, None, None]
    delta = torch.bmm(t, s["b"].float()[a].transpose(1, 2))
    r = torch.arange(s["rows"], device="cuda")
    e = torch.searchsorted(s["offsets"][1:].long(), r, right=True)
    return (s["base"].float() + delta[e, r - s["offsets"].long()[e]]).to(s["base"].dtype)


_PLAIN = {"router": _router, "router_backward": _router_backward, "activation": _activation,
          "activation_backward": _activation_backward, "combine": _combine, "combine_backward": _combine_backward,
          "adapters": _adapters}


# --------------------------------------------------------- the framework's

def _constants(s):
    names = {"situ": ("situ_beta", "situ_linear_beta"), "swiglu": (), "swiglu_bias": ("swiglu_alpha", "swiglu_beta")}
    return dict(zip(names[s["kind"]], (s["p0"], s["p1"])), activation=s["kind"], offsets=s["offsets"])


def _calls(s):
    import block_scaled_mxfp4_amd as B
    op = s["op"]
    if op == "router":
        return B.situ_moe_router(s["logits"], s["top_k"], scoring=s["scoring"], bias=s["bias"],
                                 renormalize=s["renormalize"], scale=s["scale"], mask=s["mask"], balance=s["balance"])
    if op == "router_backward":
        return B.situ_moe_router_backward(s["logits"], s["ids"], s["d_weights"], scoring=s["scoring"],
                                          renormalize=s["renormalize"], scale=s["scale"], mask=s["mask"],
                                          counts=s["counts"], d_loss=s["d_loss"])
    if op == "activation":
        if not s["keep"]:
            return B.situ_moe_activation(s["gate_up"], **_constants(s))
        h, codes, scales = B.situ_moe_activation(s["gate_up"], checkpoint=True, **_constants(s))
        return h, codes.view(F8), scales
    if op == "activation_backward":
        return B.situ_moe_activation_backward(s["d_out"], *s["kept"], recompute=True, **_constants(s))
    if op == "combine":
        return B.situ_moe_combine(s["y"], s["weights"], s["inv"], out_dtype=torch.bfloat16)
    if op == "combine_backward":
        return B.situ_moe_combine_backward(s["d_out"], s["y"], s["weights"], s["inv"])
    return B.situ_moe_adapters(s["x"], s["a"], s["b"], s["offsets"], s["ids"], base=s["base"], scales=s["scales"])


def run(state):
    return _calls(state) if own else _PLAIN[state["op"]](state)


# ------------------------------------------------------- work and 64 bits

def work(case):
    op = case["op"]
    size = 2 if case.get("type") == "bf16" else 4
    if op.startswith("router"):
        t, e, k = case["tokens"] - case["padded"], case["experts"], case["top_k"]
        rows = case["tokens"] * k
        if op == "router":
            return {"bytes": t * e * size + 6 * rows + (8 * e if case["balance"] else 0), "flops": 4 * t * e}
        return {"bytes": t * e * size + case["tokens"] * e * size + 8 * rows + 4 * e, "flops": 8 * t * e}
    if op.startswith("activation"):
        n = case["rows"] * case["inner"]
        kept = 2 * n + 8 * case["rows"] * blocks(case["inner"]) if case["keep"] else 4 * n
        if op == "activation":
            return {"bytes": 4 * n + 2 * n + (kept if case["keep"] else 0), "flops": 10 * n}
        return {"bytes": kept + 2 * n + 4 * n + 2 * n, "flops": 20 * n}
    if op.startswith("combine"):
        t, h = case["tokens"], case["hidden"]
        pairs = max(1, round(case["local"] * t * case["top_k"]))
        table = 6 * t * case["top_k"]
        if op == "combine":
            return {"bytes": pairs * h * size + 2 * t * h + table, "flops": 2 * pairs * h}
        return {"bytes": 2 * pairs * h * size + 2 * t * h + table + 4 * t * case["top_k"], "flops": 3 * pairs * h}
    rows, n, k, r = case["rows"], case["n"], case["k"], case["rank"]
    used = min(case["adapters"], case["requests"])
    return {"bytes": 2 * rows * k + 2 * rows * n * size + 2 * used * r * (n + k), "flops": 2 * rows * r * (n + k)}


def exact(case, seed):
    s = prepare(case, seed)
    op, d = case["op"], torch.float64
    if op.startswith("router"):
        t, e, k = case["tokens"], case["experts"], case["top_k"]
        z = s["logits"].to(d)
        lost = torch.isneginf(z) | torch.isnan(z)
        if s["mask"] is not None:
            lost = lost | ~s["mask"][:, None]
        live = ~lost.all(1)
        z = torch.where(live[:, None], z, 0.0).requires_grad_()
        p = torch.softmax(z, 1) if case["scoring"] == "softmax" else torch.sigmoid(z)
        if op == "router":
            left = (z if s["bias"] is None else p + s["bias"].to(d)).detach().masked_fill(lost, NOTHING)
            ids = torch.full((t, k), -1, dtype=torch.long, device="cuda")
            for j in range(k):                          # the largest that is left, the lowest of equals
                best = left.amax(1, keepdim=True)
                at = (left == best).to(torch.int8).argmax(1, keepdim=True)
                ids[:, j] = torch.where(best > NOTHING, at, -1)[:, 0]
                left.scatter_(1, at, NOTHING)
        else:
            ids = s["ids"].long()
        w = torch.where(ids < 0, 0.0, p.gather(1, ids.clamp(min=0)))
        if case["renormalize"]:
            w = w / w.sum(1, keepdim=True).clamp(min=1e-300)
        w = w * s["scale"]
        share = p / p.sum(1, keepdim=True) * live[:, None]
        hits = torch.zeros(t, e, dtype=torch.bool, device="cuda")
        hits.scatter_(1, ids.clamp(min=0), True)
        counts = (hits & live[:, None]).sum(0)
        loss = e * k * (counts.to(d) @ share.sum(0)) / max(int(counts.sum()), 1) ** 2
        if op == "router_backward":
            ((w * s["d_weights"].to(d) * live[:, None]).sum() + s["d_loss"].to(d)[0] * loss).backward()
            return z.grad
        out = ids.int(), w.detach()
        return (*out, counts.int(), share.sum(0).detach(), loss.detach().view(1)) if case["balance"] else out
    if op.startswith("activation"):
        inner, rows = case["inner"], case["rows"]
        bounds = s["offsets"].tolist()
        expert = torch.repeat_interleave(torch.arange(case["experts"], device="cuda"),
                                         torch.tensor(np.diff(bounds), device="cuda"))
        if op == "activation":
            whole = s["gate_up"].to(d)
        else:
            whole = s["kept"][0].view(F8).to(d) if case["keep"] else s["kept"][0].to(d)
            if case["keep"]:
                column = torch.arange(2 * inner, device="cuda")
                whole = whole * s["kept"][1].to(d)[:, column // inner * blocks(inner) + column % inner // 128]
        whole.requires_grad_()
        g, u = whole.split(inner, 1)
        p0, p1 = s["p0"].to(d)[expert, None], s["p1"].to(d)[expert, None]
        if case["kind"] == "situ":
            h = p0 * torch.tanh(g / p0) * torch.sigmoid(g) * p1 * torch.tanh(u / p1)
        elif case["kind"] == "swiglu":
            h = g * torch.sigmoid(g) * u
        else:
            h = g * torch.sigmoid(p0 * g) * (u + p1)
        if op == "activation_backward":
            h.backward(s["d_out"].to(d))
            return whole.grad, h.detach()
        h = h.detach()
        if not case["keep"]:
            return h
        codes, scales = [], []
        for half in (g.detach(), u.detach()):
            for c in range(0, inner, 128):
                part = half[:, c:c + 128]
                scales.append(torch.clamp(part.abs().max(dim=1).values, min=TINY) / F8_MAX)
                codes.append(part / scales[-1][:, None])
        return h, torch.cat(codes, 1), torch.stack(scales, 1)
    if op.startswith("combine"):
        t, k = case["tokens"], case["top_k"]
        out = torch.zeros(t, case["hidden"], dtype=d, device="cuda")
        dy, dw = torch.zeros(s["y"].shape, dtype=d, device="cuda"), torch.zeros(t, k, dtype=d, device="cuda")
        for j in range(k):
            tokens = torch.nonzero(s["inv"][:, j] >= 0)[:, 0]
            at = s["inv"][tokens, j].long()
            y, w = s["y"][at].to(d), s["weights"][tokens, j].to(d)
            if op == "combine":
                out[tokens] += w[:, None] * y
            else:
                g = s["d_out"][tokens].to(d)
                dy[at], dw[tokens, j] = w[:, None] * g, (g * y).sum(1)
        return out if op == "combine" else (dy, dw)
    out = s["base"].to(d)
    bounds = s["offsets"].tolist()
    for i, a in enumerate(s["ids"].tolist()):
        lo, hi = bounds[i], bounds[i + 1]
        if a >= 0 and hi > lo:
            t = s["x"][lo:hi].to(d) @ s["a"][a].to(d).t()
            out[lo:hi] += s["scales"][a].to(d) * (t @ s["b"][a].to(d).t())
    return out
