"""What the steps around the routed products refuse, on the host (no GPU needed,
no kernel is launched)."""

import ctypes
import os
import subprocess

import pytest
import torch

import block_scaled_mxfp4_amd as B

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "situ_moe.h")
FAKE = 1 << 20          # never dereferenced: every case fails on the host first
NAN, INF = float("nan"), float("inf")

STRUCTS = {"situ_moe_router_t": B.SituMoeRouter, "situ_moe_router_backward_t": B.SituMoeRouterBackward,
           "situ_moe_activation_t": B.SituMoeActivation, "situ_moe_combine_t": B.SituMoeCombine,
           "situ_moe_adapters_t": B.SituMoeAdapters}


def test_struct_layout_matches_header(tmp_path):
    lines = ['#include <stdio.h>', '#include <stddef.h>', f'#include "{HEADER}"', "int main(void) {"]
    for st, cls in STRUCTS.items():
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
        assert (ctypes.sizeof(STRUCTS[st]) if f == "size" else getattr(STRUCTS[st], f).offset) == int(v), (st, f)
        n += 1
    assert n == sum(len(c._fields_) + 1 for c in STRUCTS.values())


def call(fn, cls, base, kw):
    status = getattr(B.load(), fn)(ctypes.byref(cls(**dict(base, **kw))), None)
    return status


@pytest.mark.parametrize("fn", ["situ_moe_router", "situ_moe_router_backward", "situ_moe_activation",
                                "situ_moe_activation_backward", "situ_moe_combine", "situ_moe_combine_backward",
                                "situ_moe_adapters", "situ_moe_router_workspace", "situ_moe_adapters_workspace"])
def test_null_args(fn):
    assert getattr(B.load(), fn)(None, None) == 1


ROUTER = dict(tokens=400, experts=96, top_k=4, scoring=0, logits_dtype=B.OUT_F32, weights_dtype=B.OUT_BF16, renormalize=1,
              scale=1.0, logits_stride=96, logits=FAKE, ids=FAKE, weights=FAKE)
LOSS = dict(counts=FAKE, prob_sum=FAKE, loss=FAKE, workspace=FAKE, workspace_bytes=1 << 30)


@pytest.mark.parametrize("kw,want", [
    (dict(tokens=-1), 2), (dict(experts=0), 2), (dict(top_k=0), 2), (dict(top_k=97), 2), (dict(experts=1025, logits_stride=1025), 3),
    (dict(top_k=65), 3), (dict(tokens=(1 << 24) + 1), 3), (dict(scoring=2), 3), (dict(scoring=-1), 3), (dict(logits_dtype=2), 3),
    (dict(weights_dtype=5), 3), (dict(renormalize=2), 2), (dict(scale=NAN), 2), (dict(scale=INF), 2), (dict(bias=FAKE), 3),
    (dict(logits=None), 1), (dict(ids=None), 1), (dict(logits=FAKE + 2), 2), (dict(ids=FAKE + 1), 2), (dict(weights=FAKE + 1), 2),
    (dict(logits_stride=95), 2), (dict(logits_stride=1 << 41), 2), (dict(packed=FAKE + 2), 2),
    (dict(scoring=1, bias=FAKE + 2), 2), (dict(counts=FAKE), 1), (dict(counts=FAKE, loss=FAKE), 1),
    (dict(LOSS, workspace=None), 6), (dict(LOSS, workspace_bytes=100), 6), (dict(LOSS, workspace=FAKE + 8), 2),
    (dict(LOSS, loss=FAKE + 1), 2), (dict(LOSS, counts=FAKE + 2), 2), (dict(tokens=0, logits=None, ids=None), 0)])
def test_router_refusals(kw, want):
    assert call("situ_moe_router", B.SituMoeRouter, ROUTER, kw) == want, B.situ_moe_last_error()


def test_router_workspace():
    n = ctypes.c_uint64(7)
    fn = B.load().situ_moe_router_workspace
    assert fn(ctypes.byref(B.SituMoeRouter(**ROUTER)), ctypes.byref(n)) == 0 and n.value == 0
    sizes = []
    for tokens in (0, 1, 100, 1 << 24):
        assert fn(ctypes.byref(B.SituMoeRouter(**dict(ROUTER, **LOSS, tokens=tokens))), ctypes.byref(n)) == 0
        sizes.append(n.value)
    assert sizes[0] <= sizes[1] <= sizes[2] <= sizes[3] < 1 << 24 and sizes[2] > 0
    assert fn(ctypes.byref(B.SituMoeRouter(**ROUTER)), None) == 1
    assert fn(ctypes.byref(B.SituMoeRouter(**dict(ROUTER, top_k=200))), ctypes.byref(n)) == 2


BACK = dict(tokens=40, experts=96, top_k=4, scoring=0, logits_dtype=B.OUT_F32, out_dtype=B.OUT_F32, renormalize=1, scale=1.0,
            logits_stride=96, out_stride=96, logits=FAKE, ids=FAKE, d_weights=FAKE, counts=FAKE, d_loss=FAKE, d_logits=FAKE)


@pytest.mark.parametrize("kw,want", [
    (dict(tokens=-1), 2), (dict(top_k=97), 2), (dict(top_k=65), 3), (dict(experts=1025, logits_stride=1025, out_stride=1025), 3),
    (dict(scoring=3), 3), (dict(out_dtype=2), 3), (dict(scale=-INF), 2), (dict(counts=None), 1), (dict(d_loss=None), 1),
    (dict(counts=None, d_loss=None, d_weights=None), 1), (dict(logits=None), 1), (dict(d_logits=None), 1), (dict(ids=None), 1),
    (dict(logits=FAKE + 1), 2), (dict(d_logits=FAKE + 2), 2), (dict(out_stride=90), 2), (dict(d_weights=FAKE + 1), 2),
    (dict(ids=FAKE + 2), 2), (dict(renormalize=-1), 2), (dict(tokens=0, logits=None, d_logits=None), 0)])
def test_router_backward_refusals(kw, want):
    assert call("situ_moe_router_backward", B.SituMoeRouterBackward, BACK, kw) == want, B.situ_moe_last_error()


ACT = dict(rows=10, inner=200, experts=3, activation=0, gate_up_stride=400, h_stride=200, dh_stride=200, d_gate_up_stride=400,
           offsets=FAKE, p0=FAKE, p1=FAKE, gate_up=FAKE, h=FAKE, dh=FAKE, d_gate_up=FAKE)


@pytest.mark.parametrize("fn", ["situ_moe_activation", "situ_moe_activation_backward"])
@pytest.mark.parametrize("kw,want", [
    (dict(rows=-1), 2), (dict(inner=0), 2), (dict(inner=196), 2), (dict(experts=0), 2), (dict(experts=1025), 3),
    (dict(inner=(1 << 17) + 8), 3), (dict(rows=(1 << 24) + 1), 3), (dict(activation=3), 3), (dict(activation=-1), 3),
    (dict(offsets=None), 1), (dict(offsets=FAKE + 2), 2), (dict(p0=None), 1), (dict(p1=None), 1), (dict(p1=FAKE + 1), 2),
    (dict(activation=2, p0=None), 1), (dict(codes=FAKE), 1), (dict(scales=FAKE), 1), (dict(codes=FAKE + 4, scales=FAKE), 2),
    (dict(codes=FAKE, scales=FAKE + 2), 2), (dict(gate_up=FAKE + 8), 2), (dict(gate_up_stride=396), 2),
    (dict(gate_up_stride=404), 2), (dict(h=FAKE + 8), 2), (dict(h_stride=192), 2), (dict(rows=0, gate_up=None, h=None), 0)])
def test_activation_refusals(kw, want, fn):
    assert call(fn, B.SituMoeActivation, ACT, kw) == want, B.situ_moe_last_error()


@pytest.mark.parametrize("fn,kw,want", [
    ("", dict(gate_up=None), 1), ("", dict(h=None), 1), ("_backward", dict(gate_up=None), 1),
    ("_backward", dict(codes=FAKE, scales=FAKE), 1), ("_backward", dict(dh=None), 1), ("_backward", dict(d_gate_up=None), 1),
    ("_backward", dict(dh=FAKE + 8), 2), ("_backward", dict(dh_stride=196), 2), ("_backward", dict(d_gate_up_stride=200), 2),
    ("_backward", dict(d_gate_up=FAKE + 2), 2)])
def test_activation_directions(fn, kw, want):
    assert call("situ_moe_activation" + fn, B.SituMoeActivation, ACT, kw) == want, B.situ_moe_last_error()


COMB = dict(tokens=5, top_k=4, hidden=96, rows=20, y_dtype=B.OUT_BF16, weights_dtype=B.OUT_F32, out_dtype=B.OUT_BF16,
            y_stride=96, out_stride=96, dy_stride=96, y=FAKE, weights=FAKE, inv=FAKE, out=FAKE, dy=FAKE, d_weights=FAKE)


@pytest.mark.parametrize("fn", ["situ_moe_combine", "situ_moe_combine_backward"])
@pytest.mark.parametrize("kw,want", [
    (dict(tokens=-1), 2), (dict(rows=-1), 2), (dict(top_k=0), 2), (dict(top_k=1025), 3), (dict(hidden=0), 2), (dict(hidden=100), 2),
    (dict(hidden=(1 << 18) + 8), 3), (dict(rows=(1 << 24) + 1), 3), (dict(tokens=(1 << 24) + 1), 3), (dict(y_dtype=4), 3),
    (dict(weights_dtype=-1), 3), (dict(out_dtype=2), 3), (dict(reserved=1), 2), (dict(y=None), 1), (dict(weights=None), 1),
    (dict(inv=None), 1), (dict(out=None), 1), (dict(y=FAKE + 8), 2), (dict(inv=FAKE + 2), 2), (dict(weights=FAKE + 2), 2),
    (dict(out=FAKE + 4), 2), (dict(y_stride=88), 2), (dict(y_stride=100), 2), (dict(out_stride=92), 2),
    (dict(tokens=0, y=None, out=None), 0)])
def test_combine_refusals(kw, want, fn):
    assert call(fn, B.SituMoeCombine, COMB, kw) == want, B.situ_moe_last_error()


@pytest.mark.parametrize("kw,want", [
    (dict(dy=None, d_weights=None), 1), (dict(dy=FAKE + 8), 2), (dict(dy_stride=90), 2), (dict(d_weights=FAKE + 2), 2)])
def test_combine_backward_refusals(kw, want):
    assert call("situ_moe_combine_backward", B.SituMoeCombine, COMB, kw) == want, B.situ_moe_last_error()


ADAPT = dict(rows=20, n=96, k=128, rank=16, requests=3, adapters=2, out_dtype=B.OUT_BF16, x_stride=128, base_stride=96,
             out_stride=96, offsets=FAKE, adapter=FAKE, x=FAKE, a=FAKE, b=FAKE, base=FAKE, out=FAKE, workspace=FAKE,
             workspace_bytes=1 << 30)
LARGE = dict(rows=1000)          # has a workspace


@pytest.mark.parametrize("kw,want", [
    (dict(rows=-1), 2), (dict(n=0), 2), (dict(n=100), 2), (dict(k=4), 2), (dict(k=132), 2), (dict(rank=0), 2), (dict(rank=12), 2),
    (dict(rank=264), 3), (dict(n=(1 << 18) + 8), 3), (dict(k=(1 << 18) + 8), 3), (dict(rows=(1 << 24) + 1), 3),
    (dict(requests=0), 2), (dict(adapters=0), 2), (dict(requests=(1 << 20) + 1), 3), (dict(adapters=(1 << 20) + 1), 3),
    (dict(out_dtype=2), 3), (dict(reserved=4), 2), (dict(offsets=None), 1), (dict(adapter=None), 1), (dict(x=None), 1),
    (dict(a=None), 1), (dict(b=None), 1), (dict(out=None), 1), (dict(offsets=FAKE + 1), 2), (dict(adapter=FAKE + 2), 2),
    (dict(ranks=FAKE + 2), 2), (dict(scales=FAKE + 1), 2), (dict(x=FAKE + 8), 2), (dict(a=FAKE + 2), 2), (dict(b=FAKE + 8), 2),
    (dict(base=FAKE + 8), 2), (dict(base_stride=95), 2), (dict(out=FAKE + 2), 2), (dict(out_stride=100), 2),
    (dict(x_stride=120), 2), (dict(x_stride=1 << 41), 2), (dict(LARGE, workspace=None), 6), (dict(LARGE, workspace_bytes=8), 6),
    (dict(LARGE, workspace=FAKE + 4), 2), (dict(rows=0, x=None, out=None, workspace=None), 0)])
def test_adapters_refusals(kw, want):
    assert call("situ_moe_adapters", B.SituMoeAdapters, ADAPT, kw) == want, B.situ_moe_last_error()


def test_adapters_workspace():
    n = ctypes.c_uint64()
    fn = B.load().situ_moe_adapters_workspace
    for rows, k, rank in ((0, 128, 16), (1, 8, 8), (64, 3584, 16), (8192, 3584, 32), (1 << 24, 1 << 18, 256)):
        assert fn(ctypes.byref(B.SituMoeAdapters(**dict(ADAPT, rows=rows, k=k, rank=rank))), ctypes.byref(n)) == 0
        assert n.value % (4 * max(rows, 1) * rank) == 0 and n.value <= 64 * 4 * rows * rank
        assert rows < 1000 or n.value > 0
    assert fn(ctypes.byref(B.SituMoeAdapters(**ADAPT)), None) == 1


@pytest.mark.parametrize("make", [
    lambda x: B.situ_moe_router(x, 2), lambda x: B.situ_moe_router_backward(x, x), lambda x: B.situ_moe_activation(x.bfloat16()),
    lambda x: B.situ_moe_activation_backward(x.bfloat16(), x), lambda x: B.situ_moe_combine(x, x, x),
    lambda x: B.situ_moe_combine_backward(x, x, x, x), lambda x: B.situ_moe_adapters(x.bfloat16(), x, x, x, x)])
def test_host_tensors_are_refused(make):
    with pytest.raises(B.SituMoeError) as e:
        make(torch.zeros(4, 16))
    assert e.value.status_name == "SITU_E_DEVICE"
