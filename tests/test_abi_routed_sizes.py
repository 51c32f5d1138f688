"""Sizes at the ends of their types in the calls of the steps around the routed
products, on the host (no GPU needed, no kernel is launched)."""

import ctypes

import pytest
import torch

import block_scaled_mxfp4_amd as B
from test_abi_grouped import _Fake, _status
from test_abi_routed import ADAPT

BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32
MANY = (1 << 31) + 4


@pytest.fixture
def fakes(monkeypatch):
    if torch.cuda.is_available():
        pytest.skip("a GPU is present: the addresses of these tensors are not memory")
    from block_scaled_mxfp4_amd import routed
    routed._first()
    monkeypatch.setattr(routed, "_device", lambda: 0)
    monkeypatch.setattr(routed, "_raw_stream", lambda dev: 0)
    return _Fake


def test_sizes_past_32_bits(fakes):
    """They are refused with this library's error, also where a workspace is sized first."""
    def router(tokens, **kw):
        return B.situ_moe_router(fakes(F32, tokens, 8), 2, ids=fakes(I32, tokens, 2), weights=fakes(BF, tokens, 2), **kw)

    def adapters(rows, k, n, requests, rank=8):
        return B.situ_moe_adapters(fakes(BF, rows, k), fakes(BF, 2, rank, k), fakes(BF, 2, n, rank), fakes(I32, requests + 1),
                                   fakes(I32, requests), out=fakes(BF, rows, n))

    loss = dict(counts=fakes(I32, 8), prob_sum=fakes(F32, 8), loss=fakes(F32, 1))
    assert _status(lambda: router(4)) == "SITU_E_DEVICE"                        # the fakes pass where sizes do
    assert _status(lambda: router(4, **loss)) == "SITU_E_DEVICE"
    assert _status(lambda: adapters(4, 64, 32, 2)) == "SITU_E_DEVICE"
    wide = fakes(BF, 4, 1 << 32)
    for call in (lambda: router(MANY), lambda: router(MANY, **loss),
                 lambda: B.situ_moe_router_backward(fakes(F32, MANY, 8), fakes(I32, MANY, 2), fakes(F32, MANY, 2),
                                                    out=fakes(F32, MANY, 8)),
                 lambda: B.situ_moe_activation(fakes(BF, MANY, 32), activation="swiglu", out=fakes(BF, MANY, 16)),
                 lambda: B.situ_moe_activation(wide, activation="swiglu", out=fakes(BF, 4, 1 << 31)),
                 lambda: B.situ_moe_activation_backward(fakes(BF, MANY, 16), fakes(BF, MANY, 32), activation="swiglu",
                                                        out=fakes(BF, MANY, 32)),
                 lambda: B.situ_moe_combine(fakes(BF, MANY, 8), fakes(BF, 3, 2), fakes(I32, 3, 2), out=fakes(BF, 3, 8)),
                 lambda: B.situ_moe_combine_backward(fakes(BF, 3, 8), fakes(BF, MANY, 8), fakes(BF, 3, 2), fakes(I32, 3, 2),
                                                     dy=fakes(BF, MANY, 8), d_weights=fakes(F32, 3, 2)),
                 lambda: adapters(MANY, 64, 32, 2), lambda: adapters(4, 1 << 31, 32, 2), lambda: adapters(4, 64, 1 << 31, 2),
                 lambda: adapters(4, 64, 32, MANY), lambda: adapters(4, 64, 32, 2, rank=1 << 31)):
        assert _status(call) == "SITU_E_UNSUPPORTED"


def test_adapters_workspace_of_many_requests():
    """The rule that goes by rows and requests does not leave 32 bits: more requests than the call takes ask for no more."""
    n = ctypes.c_uint64()
    sizes = []
    for requests in (1 << 20, (1 << 30) - 1, 1 << 30, (1 << 31) - 1):
        args = B.SituMoeAdapters(**dict(ADAPT, rows=512, requests=requests))
        assert B.load().situ_moe_adapters_workspace(ctypes.byref(args), ctypes.byref(n)) == 0
        sizes.append(n.value)
    assert sizes == [0] * 4
