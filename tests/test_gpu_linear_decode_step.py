"""Decode steps of linear attention over offsets: sequences of one token or none,
padding rows, and steps of unequal counts through the layer, against the
recurrence in 64 bits.

Tolerances.  One token: S = a S_0 + v k^T with e^g of two units in the last place
(2^-22) and two roundings, below 2^-21 of the terms' absolute values (`weight`);
an output sums 128 such terms in fp32 (at most 11 roundings each) and is rounded
to bf16: 2^-8 of it and 2^-19 of its weight.  Several tokens run in chunks, whose
terms are two bf16 parts in the output (2^-14 of the weight with the fp32 sums)
and three in the state, over a handful of tokens (2^-17).
"""
import pytest
import torch

import attention_attn_varlen_gb300 as av
from attention_attn_varlen_gb300.attention import LinearAttention, PagePool
from _step_reference import cu_of, linear

pytestmark = pytest.mark.gpu


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _decay(Hkv):
    return (-(2.0 ** (-8.0 * torch.arange(1, Hkv + 1, dtype=torch.float64) / Hkv))).float()


def _qkv(gen, rows, Hq, Hkv, D):
    """q, k, v as views of one packed projection, on the CPU and the GPU."""
    x = torch.randn(rows, Hq + 2 * Hkv, D, generator=gen).to(torch.bfloat16)
    cut = lambda y: (y[:, :Hq], y[:, Hq:Hq + Hkv], y[:, Hq + Hkv:])  # noqa: E731
    return cut(x), cut(x.cuda())


def _close(got, ref, weight, one, what):
    err = (got.double().cpu() - ref).abs()
    assert (err <= 2.0 ** -8 * ref.abs() + 2.0 ** (-19 if one else -14) * weight).all(), what


@pytest.mark.parametrize("B,Hq,Hkv,D", [(1, 1, 1, 64), (4, 4, 2, 128), (130, 6, 2, 64), (61, 5, 1, 128)])
@pytest.mark.parametrize("states", ["none", "fresh", "cached"])
def test_offsets_of_at_most_one_token_each(B, Hq, Hkv, D, states):
    gen = torch.Generator().manual_seed(B + D)
    new = [1] if B == 1 else torch.randint(0, 2, (B,), generator=gen).tolist()
    T, pad = sum(new), 3
    (q, k, v), dev = _qkv(gen, T + pad, Hq, Hkv, D)
    dev[0][T:] = float("nan")                            # rows behind the last sequence are not read or written
    g, cu = _decay(Hkv), cu_of(new)
    state = torch.randn(B + 2, Hkv, D, D, generator=gen)
    slots = torch.randperm(B + 2, generator=gen)[:B].to(torch.int32)
    slots[1::7] = -1
    past = torch.tensor([b % 3 for b in range(B)], dtype=torch.int32)
    sd = state.cuda()
    kw = dict(state_cache=sd, state_slots=slots.cuda()) if states != "none" else {}
    if states == "cached":
        kw["context_lens"] = past.cuda()
    out = torch.full((T + pad, Hq, D), 7.0, dtype=torch.bfloat16, device="cuda")
    av.get_last_device_error()
    av.linear_attn_varlen_fwd(*dev, g.cuda(), cu.cuda(), 1, 0.3, out=out, **kw)
    starts = [state[slots[b]].double() if states == "cached" and past[b] and slots[b] >= 0 else None for b in range(B)]
    ref, finals, weight = linear(q[:T], k[:T], v[:T], g, cu, 0.3, starts)
    _close(out[:T], ref, weight, True, "out")
    assert out[T:].eq(7.0).all()
    got, want = sd.cpu(), state.clone()
    for b in range(B):
        if states != "none" and new[b] and slots[b] >= 0:
            S, A = finals[b]
            assert ((got[slots[b]].double() - S).abs() <= 2.0 ** -21 * A + 1e-30).all(), b
            want[slots[b]] = got[slots[b]]
    assert torch.equal(got, want)                        # every other slot as it was
    assert av.get_last_device_error()[0] == 0


def test_a_token_for_every_sequence_gives_the_bits_of_the_recurrent_form():
    B, H, D = 9, 2, 128
    gen = torch.Generator().manual_seed(1)
    _, dev = _qkv(gen, B, H, H, D)
    a = torch.randn(B, H, D, D, generator=gen).cuda()
    b, slots, g = a.clone(), _i32(list(range(B))), _decay(H).cuda()
    x = av.linear_attn_varlen_fwd(*dev, g, cu_of([1] * B).cuda(), 1, state_cache=a, state_slots=slots,
                                  context_lens=torch.ones_like(slots))
    y = av.linear_attn_decode(*dev, g, b, slots)
    assert torch.equal(x, y) and torch.equal(a, b)


def test_longer_sequences_and_bad_offsets_are_reported():
    H, D = 2, 64
    gen = torch.Generator().manual_seed(2)
    _, dev = _qkv(gen, 6, H, H, D)
    g, start = _decay(H).cuda(), torch.randn(3, H, D, D, generator=gen).cuda()
    ones, slots = _i32([1, 1, 1]), _i32([0, 1, 2])

    def call(cu, n=3):
        s, out = start.clone(), torch.full((6, H, D), 7.0, dtype=torch.bfloat16, device="cuda")
        av.linear_attn_varlen_fwd(*dev, g, _i32(cu), 1, state_cache=s, state_slots=slots[:n], context_lens=ones[:n],
                                  out=out)
        return s, out, av.get_last_device_error()[0]

    av.get_last_device_error()
    s, out, status = call([0, 1, 4, 5])                  # three tokens in the middle: cut to the first
    s1, out1, status1 = call([0, 1, 2, 2])
    assert status == 6 and status1 == 0 and torch.equal(s[:2], s1[:2]) and torch.equal(out[:2], out1[:2])
    assert out[2:4].eq(7.0).all() and not out[4].eq(7.0).all()
    s, out, status = call([0, 1, 0, 90])                 # decreasing, and past the tokens
    assert status == 6 and torch.equal(s[1:], start[1:]) and out[1:].eq(7.0).all()
    s, out, status = call([-1, 0], 1)
    assert status == 6 and torch.equal(s, start) and out.eq(7.0).all()


@pytest.mark.parametrize("new,pad", [([2, 0], 0), ([3, 1, 0, 0], 0), ([2, 0, 1], 0), ([1, 0, 1, 1], 1), ([1, 0, 1, 1], 0),
                                     ([0, 1], 1), ([1, 1, 1], 2), ([2, 2], 0), ([0, 0, 4, 0], 0)])
def test_the_layer_goes_by_the_steps_counts(new, pad):
    """Every entry has a slot, those without a token too: their states stay, and the tokens
    reach the entries they belong to."""
    B, Hq, Hkv, D = len(new), 4, 2, 64
    gen = torch.Generator().manual_seed(7)
    g = _decay(Hkv)
    pool = PagePool(20, 16, B, 4)
    layer = LinearAttention(Hq, D, D ** -0.5, Hkv, g.cuda())
    state = torch.randn(B, Hkv, D, D, generator=gen)
    layer.state_cache = state.cuda()
    past = [3] + [b % 2 * 5 for b in range(1, B)]        # some have no past: they start from zero
    pool.grow(_i32(past), sum(past))
    T = sum(new)
    (q, k, v), dev = _qkv(gen, T + pad, Hq, Hkv, D)
    t = pool.grow(_i32(new), T + pad)
    av.get_last_device_error()
    y = layer(*dev, pool.context(t, False, max(new), 64, state_slots=_i32(list(range(B)))))
    starts = [state[b].double() if past[b] else None for b in range(B)]
    ref, finals, weight = linear(q[:T], k[:T], v[:T], g, cu_of(new), D ** -0.5, starts)
    _close(y[:T], ref, weight, max(new) == 1, "out")
    got = layer.state_cache.cpu()
    for b in range(B):
        if new[b]:
            assert ((got[b].double() - finals[b][0]).abs() <= 2.0 ** -17 * finals[b][1]).all(), b
        else:
            assert torch.equal(got[b], state[b]), b
    assert av.get_last_device_error()[0] == 0
