"""Calls of the steps around the routed products as a caller may make them: no
rows, inputs that require grad, raw stream handles, and what is refused of
tensors on the GPU (no kernel is launched)."""

import pytest
import torch

import block_scaled_mxfp4_amd as B

pytestmark = pytest.mark.gpu

BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32


def zeros(*shape, dtype=BF):
    return torch.zeros(*shape, dtype=dtype, device="cuda")


def refused(status, call, *args, **kw):
    with pytest.raises(B.SituMoeError) as e:
        call(*args, **kw)
    assert e.value.status_name == status, e.value


def test_no_rows():
    off = zeros(4, dtype=I32)
    one = torch.ones(3, device="cuda")
    ids, w, packed, counts, prob_sum, loss = B.situ_moe_router(zeros(0, 8, dtype=F32), 2, balance=True, packed=True)
    assert ids.shape == w.shape == packed.shape == (0, 2) and not counts.any() and not prob_sum.any() and loss.item() == 0
    d = B.situ_moe_router_backward(zeros(0, 8, dtype=F32), zeros(0, 2, dtype=I32), zeros(0, 2, dtype=F32))
    assert d.shape == (0, 8)
    h, codes, scales = B.situ_moe_activation(zeros(0, 64), offsets=off, situ_beta=one, situ_linear_beta=one, checkpoint=True)
    assert h.shape == (0, 32) and codes.shape == (0, 64) and scales.shape == (0, 2)
    d, h = B.situ_moe_activation_backward(zeros(0, 32), codes, scales, offsets=off, situ_beta=one, situ_linear_beta=one,
                                          recompute=True)
    assert d.shape == (0, 64) and h.shape == (0, 32)
    assert B.situ_moe_combine(zeros(0, 64), zeros(0, 2), zeros(0, 2, dtype=I32)).shape == (0, 64)
    # tokens, but no local row
    inv = torch.full((3, 2), -1, dtype=I32, device="cuda")
    out = B.situ_moe_combine(zeros(0, 64), torch.ones(3, 2, device="cuda"), inv)
    assert out.shape == (3, 64) and not out.any()
    dy, dw = B.situ_moe_combine_backward(torch.ones(3, 64, device="cuda"), zeros(0, 64), torch.ones(3, 2, device="cuda"), inv)
    assert dy.shape == (0, 64) and not dw.any()
    out = B.situ_moe_adapters(zeros(0, 64), zeros(2, 8, 64), zeros(2, 32, 8), off, zeros(3, dtype=I32))
    assert out.shape == (0, 32)
    # a group without rows among others, all rows behind the last group
    assert B.situ_moe_activation(zeros(5, 64), activation="swiglu", offsets=off).shape == (5, 32)


def test_inputs_that_require_grad():
    x = torch.randn(6, 64, device="cuda", dtype=BF, requires_grad=True)
    z = torch.randn(6, 16, device="cuda", requires_grad=True)
    outs = [*B.situ_moe_router(z, 2, balance=True), B.situ_moe_activation(x, activation="swiglu"),
            B.situ_moe_combine(x, torch.ones(3, 2, device="cuda", requires_grad=True),
                               torch.arange(6, dtype=I32, device="cuda").view(3, 2)),
            B.situ_moe_adapters(x, zeros(1, 8, 64), zeros(1, 32, 8), torch.tensor([0, 6], dtype=I32, device="cuda"),
                                zeros(1, dtype=I32))]
    assert not any(t.requires_grad for t in outs)


def test_default_streams_handle():
    """Handle 0 is the default stream: what it computes first is waited for."""
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    side = torch.cuda.Stream()
    for i in range(3):
        late = torch.randn(1 << 25, generator=g, device="cuda").sort().values
        x = late[::(1 << 25) // (64 * 256)][:64 * 256].view(64, 256).to(BF)
        want = None
        with torch.cuda.stream(side):
            got = B.situ_moe_activation(x, activation="swiglu", stream=0)
        torch.cuda.synchronize()
        want = B.situ_moe_activation(x, activation="swiglu")
        assert torch.equal(got, want), i


def test_scalars_and_flat_tables():
    z = torch.randn(9, 24, device="cuda")
    ids, _, counts, _, loss = B.situ_moe_router(z, 3, balance=True)
    a = B.situ_moe_router_backward(z, ids, counts=counts, d_loss=torch.ones(1, device="cuda"))
    b = B.situ_moe_router_backward(z, ids, counts=counts, d_loss=torch.ones((), device="cuda"))
    assert torch.equal(a, b)
    # a scale of zero and below
    _, w = B.situ_moe_router(z, 3, scale=0.0)
    assert not w.any()
    up, down = (B.situ_moe_router(z, 3, scale=s, weights_dtype=F32)[1] for s in (1.5, -1.5))
    assert torch.equal(up, -down)


def test_router_refusals():
    z = zeros(4, 16, dtype=F32)
    refused("SITU_E_BAD_SHAPE", B.situ_moe_router, z.to(torch.float16), 2)
    refused("SITU_E_BAD_SHAPE", B.situ_moe_router, z[0], 2)
    refused("SITU_E_BAD_SHAPE", B.situ_moe_router, z.t(), 2)
    refused("SITU_E_BAD_SHAPE", B.situ_moe_router, z, 17)
    refused("SITU_E_BAD_SHAPE", B.situ_moe_router, z, 0)
    refused("SITU_E_UNSUPPORTED", B.situ_moe_router, z, 2, scoring="relu")
    refused("SITU_E_UNSUPPORTED", B.situ_moe_router, z, 2, bias=zeros(16, dtype=F32))
    refused("SITU_E_BAD_SHAPE", B.situ_moe_router, z, 2, scoring="sigmoid", bias=zeros(15, dtype=F32))
    refused("SITU_E_BAD_SHAPE", B.situ_moe_router, z, 2, mask=zeros(5, dtype=torch.bool))
    refused("SITU_E_BAD_SHAPE", B.situ_moe_router, z, 2, mask=zeros(4, dtype=I32))
    refused("SITU_E_BAD_SHAPE", B.situ_moe_router, z, 2, ids=zeros(4, 2, dtype=torch.int64))
    refused("SITU_E_UNSUPPORTED", B.situ_moe_router, z, 2, weights_dtype=torch.float16)
    refused("SITU_E_BAD_SHAPE", B.situ_moe_router, z, 2, scale=float("nan"))
    refused("SITU_E_UNSUPPORTED", B.situ_moe_router, z, 2, scale=1e39)
    refused("SITU_E_WORKSPACE", B.situ_moe_router, zeros(400, 16, dtype=F32), 2, balance=True,
            workspace=zeros(64, dtype=torch.uint8))
    ids = zeros(4, 2, dtype=I32)
    refused("SITU_E_NULL_ARG", B.situ_moe_router_backward, z, ids)
    refused("SITU_E_NULL_ARG", B.situ_moe_router_backward, z, ids, counts=zeros(16, dtype=I32))
    refused("SITU_E_NULL_ARG", B.situ_moe_router_backward, z, None, zeros(4, 2, dtype=F32))
    refused("SITU_E_BAD_SHAPE", B.situ_moe_router_backward, z, ids, zeros(4, 3, dtype=F32))
    refused("SITU_E_BAD_SHAPE", B.situ_moe_router_backward, z, zeros(3, 2, dtype=I32), zeros(3, 2, dtype=F32))


def test_activation_refusals():
    x = zeros(4, 64)
    one = torch.ones(1, device="cuda")
    refused("SITU_E_NULL_ARG", B.situ_moe_activation, x)
    refused("SITU_E_NULL_ARG", B.situ_moe_activation, x, activation="swiglu_bias", swiglu_alpha=one)
    refused("SITU_E_UNSUPPORTED", B.situ_moe_activation, x, activation="gelu")
    refused("SITU_E_BAD_SHAPE", B.situ_moe_activation, zeros(4, 40), activation="swiglu")
    refused("SITU_E_BAD_SHAPE", B.situ_moe_activation, x.float(), activation="swiglu")
    refused("SITU_E_BAD_SHAPE", B.situ_moe_activation, zeros(4, 72)[:, 4:68], activation="swiglu")    # 8-byte aligned rows
    refused("SITU_E_BAD_SHAPE", B.situ_moe_activation, zeros(4, 68)[:, :64], activation="swiglu")
    refused("SITU_E_BAD_SHAPE", B.situ_moe_activation, x, situ_beta=torch.ones(2, device="cuda"), situ_linear_beta=one)
    refused("SITU_E_BAD_SHAPE", B.situ_moe_activation, x, activation="swiglu", codes=zeros(4, 32, dtype=torch.uint8))
    refused("SITU_E_BAD_SHAPE", B.situ_moe_activation, x, activation="swiglu", offsets=zeros(1, dtype=I32))
    refused("SITU_E_BAD_SHAPE", B.situ_moe_activation_backward, zeros(4, 32), zeros(4, 32), activation="swiglu")
    refused("SITU_E_BAD_SHAPE", B.situ_moe_activation_backward, zeros(4, 32), x, zeros(4, 2, dtype=F32), activation="swiglu")
    refused("SITU_E_BAD_SHAPE", B.situ_moe_activation_backward, zeros(4, 32), zeros(4, 64, dtype=torch.uint8),
            zeros(4, 1, dtype=F32), activation="swiglu")


def test_combine_refusals():
    y, w, inv = zeros(6, 64), zeros(3, 2), zeros(3, 2, dtype=I32)
    refused("SITU_E_BAD_SHAPE", B.situ_moe_combine, zeros(6, 60), w, inv)
    refused("SITU_E_BAD_SHAPE", B.situ_moe_combine, y, w, zeros(5, dtype=I32))
    refused("SITU_E_BAD_SHAPE", B.situ_moe_combine, y, w.to(torch.float16), inv)
    refused("SITU_E_BAD_SHAPE", B.situ_moe_combine, y, w, inv.long())
    refused("SITU_E_NULL_ARG", B.situ_moe_combine, y, w, None)
    refused("SITU_E_UNSUPPORTED", B.situ_moe_combine, y, w, inv, out_dtype=torch.float16)
    refused("SITU_E_BAD_SHAPE", B.situ_moe_combine, y, w, inv, out=zeros(3, 64, dtype=F32), out_dtype=BF)
    refused("SITU_E_BAD_SHAPE", B.situ_moe_combine_backward, zeros(2, 64), y, w, inv)
    refused("SITU_E_BAD_SHAPE", B.situ_moe_combine_backward, zeros(3, 64), y, w, inv, dy=zeros(6, 64, dtype=F32))


def test_adapters_refusals():
    x, a, b = zeros(4, 64), zeros(2, 8, 64), zeros(2, 32, 8)
    off, ids = torch.tensor([0, 4], dtype=I32, device="cuda"), zeros(1, dtype=I32)
    refused("SITU_E_BAD_SHAPE", B.situ_moe_adapters, x, zeros(2, 8, 72), b, off, ids)
    refused("SITU_E_BAD_SHAPE", B.situ_moe_adapters, x, a, zeros(3, 32, 8), off, ids)
    refused("SITU_E_BAD_SHAPE", B.situ_moe_adapters, x, a, b, off, zeros(2, dtype=I32))
    refused("SITU_E_BAD_SHAPE", B.situ_moe_adapters, x, zeros(2, 12, 64), zeros(2, 32, 12), off, ids)
    refused("SITU_E_UNSUPPORTED", B.situ_moe_adapters, x, zeros(2, 264, 64), zeros(2, 32, 264), off, ids)
    refused("SITU_E_NULL_ARG", B.situ_moe_adapters, x, a, b, None, ids)
    refused("SITU_E_BAD_SHAPE", B.situ_moe_adapters, x, a, b, off, ids, base=zeros(4, 32, dtype=F32), out=zeros(4, 32))
    refused("SITU_E_BAD_SHAPE", B.situ_moe_adapters, x, a, b, off, ids, scales=zeros(3, dtype=F32))
    refused("SITU_E_BAD_SHAPE", B.situ_moe_adapters, x, a, b, off, ids, ranks=zeros(2, dtype=torch.int64))
    refused("SITU_E_BAD_SHAPE", B.situ_moe_adapters, x, a, b, zeros(1, dtype=I32), zeros(0, dtype=I32))
    many = zeros(600, 64)
    refused("SITU_E_WORKSPACE", B.situ_moe_adapters, many, a, b, torch.tensor([0, 600], dtype=I32, device="cuda"), ids,
            workspace=zeros(64, dtype=torch.uint8))
