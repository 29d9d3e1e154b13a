"""The step operators on a stream of their own: what they allocate must not be
memory that the current stream still works on."""
import pytest
import torch

import attention_attn_varlen_gb300 as av
from _step_reference import cu_of

pytestmark = pytest.mark.gpu


def _i32(*x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _linear(B=3, T=600, H=4, D=64):
    gen = torch.Generator(device="cuda").manual_seed(1)
    q, k, v = (torch.randn(T, H, D, generator=gen, device="cuda").bfloat16() for _ in range(3))
    g, cu, slots, ones = torch.full((H,), -0.1, device="cuda"), cu_of([200] * B).cuda(), _i32(0, 1, 2), _i32(1, 1, 1)
    state = torch.randn(B, H, D, D, generator=gen, device="cuda")

    def prompt(stream):
        s = state.clone()
        torch.cuda.synchronize()
        return lambda: (av.linear_attn_varlen_fwd(q, k, v, g, cu, 200, state_cache=s, state_slots=slots,
                                                  context_lens=ones, stream=stream), s)

    def decode(stream):
        s = state.clone()
        torch.cuda.synchronize()
        return lambda: (av.linear_attn_decode(q[:B], k[:B], v[:B], g, s, slots, stream=stream), s)

    return prompt, decode


def _rope(N=500, H=4, D=64):
    gen = torch.Generator(device="cuda").manual_seed(2)
    q, k = (torch.randn(N, H, D, generator=gen, device="cuda").bfloat16() for _ in range(2))
    pos, inv = torch.arange(N, dtype=torch.int32, device="cuda"), torch.rand(D // 2, generator=gen, device="cuda")
    return lambda stream: lambda: av.rope_store_kvcache(q, k, None, pos, inv, return_k=True, stream=stream)


def _tables(B=40, M=50, T=20000):
    lens, new = torch.arange(B, dtype=torch.int32, device="cuda") * 5, torch.full((B,), 300, device="cuda").int()
    table = torch.arange(B * M, dtype=torch.int32, device="cuda").view(B, M)
    free = torch.arange(2 * B * M, dtype=torch.int32, device="cuda").roll(B * M)    # the other half of the pool first

    def make(stream):
        pool = [lens.clone(), table.clone(), free.clone(), _i32(B * M)]
        torch.cuda.synchronize()

        def call():
            t = av.step_tables(None, new, *pool, 16, T, stream=stream)
            av.trim_pages(None, t.context_lens, *pool, 16, stream=stream)
            return (*t, *pool[:3])
        return call
    return make


@pytest.mark.parametrize("make", ["prompt", "decode", "rope", "tables"])
def test_allocations_on_another_stream(make):
    make = {"prompt": lambda: _linear()[0], "decode": lambda: _linear()[1], "rope": _rope, "tables": _tables}[make]()
    want = [x.clone() for x in make(None)()]
    side = torch.cuda.Stream()
    call = make(side)
    torch.cuda.empty_cache()
    # blocks of the outputs' and the workspace's sizes that the current stream frees while it is still to write them
    taken = [torch.empty_like(x) for x in want] + [torch.empty(n, dtype=torch.uint8, device="cuda")
                                                   for n in (512, 4096, 1 << 16, 1 << 18, 1 << 20, 1 << 21)]
    torch.cuda.synchronize()
    torch.cuda._sleep(200_000_000)                  # about 0.1 s
    for x in taken:
        x.view(torch.uint8).fill_(0xA5)
    del taken, x
    got = call()
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    assert av.get_last_device_error()[0] == 0
