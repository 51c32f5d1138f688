"""Calls of the FP8 and grouped products as a caller may make them: streams
given by their raw handles."""

import pytest
import torch

import block_scaled_mxfp4_amd as B
from block_scaled_mxfp4_amd import grouped

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def test_stream_handles():
    """The default stream's raw handle is 0; it stays the default stream."""
    grouped._first()
    dev = torch.cuda.current_device()
    device = torch.device("cuda", dev)
    side = torch.cuda.Stream()
    assert torch.cuda.default_stream().cuda_stream == 0
    assert grouped._Place(dev, 0).handle == 0
    assert grouped._Place(dev, side.cuda_stream).handle == side.cuda_stream
    assert grouped._Place(dev, side).handle == side.cuda_stream
    with torch.cuda.stream(side):
        assert grouped._Place(dev, 0).handle == 0
        assert grouped._Place(dev, None).handle == side.cuda_stream
        assert B._torch_stream(0, device).cuda_stream == 0
    assert B._torch_stream(side.cuda_stream, device).cuda_stream == side.cuda_stream


def test_layer_on_the_default_streams_handle(monkeypatch):
    """The layer's one-call form hands handle 0 on as the default stream."""
    seen = []
    monkeypatch.setattr(B, "situ_moe_run", lambda plan, tensors, workspace, stream: seen.append(stream.cuda_stream))
    T, H, I, E = 4, 256, 64, 8
    u8 = dict(dtype=torch.uint8, device="cuda")
    f32 = dict(dtype=torch.float32, device="cuda")
    args = dict(hidden_states=torch.zeros(T, H, dtype=BF, device="cuda"),
                topk_ids=torch.zeros(T, 2, dtype=torch.int32, device="cuda"),
                topk_weights=torch.zeros(T, 2, dtype=BF, device="cuda"),
                w1=torch.zeros(E, 2 * I, H // 2, **u8), w1_scale=torch.zeros(E, 2 * I, H // 32, **u8),
                w2=torch.zeros(E, H, I // 2, **u8), w2_scale=torch.zeros(E, H, I // 32, **u8),
                situ_beta=torch.ones(E, **f32), situ_linear_beta=torch.ones(E, **f32), num_experts=E,
                local_expert_offset=0, local_num_experts=E, intermediate_size=I)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        for stream in (0, side.cuda_stream, side, None):
            B.situ_moe(stream=stream, **args)
    assert seen == [0] + [side.cuda_stream] * 3


def test_product_on_the_default_streams_handle():
    """A product given handle 0 waits for what the default stream computes first."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(40)
    w = torch.randn(1, 64, 512, generator=gen, device="cuda").to(BF)
    for i in range(4):
        x = torch.zeros(300, 512, dtype=BF, device="cuda")
        late = torch.randn(1 << 26, generator=gen, device="cuda").sort().values      # keeps the default stream busy
        x.copy_(late[::(1 << 26) // (300 * 512)][:300 * 512].view(300, 512))
        got = B.situ_moe_grouped_matmul(x, w, stream=0)
        assert torch.equal(got, B.situ_moe_grouped_matmul(x, w)), i
