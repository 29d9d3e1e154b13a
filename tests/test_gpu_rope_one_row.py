"""Positions of several axes that are one row expanded (text tokens of a model with
several axes): every axis reads that row."""
import pytest
import torch

import attention_attn_varlen_gb300 as av
from attention_attn_varlen_gb300.attention import Attention, AttentionContext, Rotary

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("N", [1, 77])
@pytest.mark.parametrize("D,inter", [(128, False), (10, True)])
def test_one_row_for_every_axis(N, D, inter):
    gen = torch.Generator(device="cuda").manual_seed(N)
    q, k = (torch.randn(N, h, D, generator=gen, device="cuda").bfloat16() for h in (4, 2))
    pos = torch.randint(0, 1 << 20, (N,), generator=gen, device="cuda").int()
    inv = torch.rand(D // 2, generator=gen, device="cuda")
    axis = bytes(i % 3 for i in range(D // 2))
    call = lambda p: av.rope_store_kvcache(q, k, None, p, inv, pair_axis=axis, interleaved=inter)  # noqa: E731
    for a, b in zip(call(pos.expand(3, N)), call(pos.expand(3, N).contiguous())):
        assert torch.equal(a, b)
    with pytest.raises((ValueError, av.AttnError)):      # an axis that does not exist, in either form
        av.rope_store_kvcache(q, k, None, pos.expand(2, N), inv, pair_axis=axis)
    with pytest.raises((ValueError, av.AttnError)):
        av.rope_store_kvcache(q, k, None, pos.expand(2, N).contiguous(), inv, pair_axis=axis)


def test_through_a_layer():
    gen = torch.Generator(device="cuda").manual_seed(8)
    N, H, D = 40, 2, 64
    q, k, v = (torch.randn(N, H, D, generator=gen, device="cuda").bfloat16() for _ in range(3))
    pos = torch.arange(N, dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, N], dtype=torch.int32, device="cuda")
    inv = torch.rand(D // 2, generator=gen, device="cuda")
    layers = [Attention(H, D, D ** -0.5, H, rotary=Rotary(inv, axis)) for axis in (None, bytes(i % 3 for i in range(D // 2)))]
    ctx = lambda p: AttentionContext(True, cu_seqlens_q=cu, cu_seqlens_k=cu, max_seqlen_q=N, max_seqlen_k=N, positions=p)  # noqa: E731
    assert torch.equal(layers[0](q, k, v, ctx(pos)), layers[1](q, k, v, ctx(pos.expand(3, N))))
    assert av.get_last_device_error()[0] == 0
