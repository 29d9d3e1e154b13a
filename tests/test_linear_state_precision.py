"""What of the fp32 states of linear attention is kept through chunks, segments and
many steps: tolerances that terms of two bf16 parts instead of three, or e^(64 g)
without its part below fp32, do not meet.

One token alone reaches each value dimension (v is 1 there, 0 elsewhere; k is 1),
so S[dv, :] is e^((T - 1 - j) g) for its token j: sums do not hide the terms.  A
term's three parts add up to the fp32 weight itself, so relative to the state:
  the weight     fp32 exponential, two units in the last place (2^-22), of an
                 argument rounded to fp32 (2^-24 of it), the product and the
                 sum rounded (2^-23 together)
  each chunk     S e^(64 g) rounded (2^-24); e^(64 g) itself is off by 2^-23 of
                 its argument where that is above -0.3, else as the weight
  each segment   the same product once more, with e^(seg g) as the weight
Two parts are off by up to 2^-16.5 for some of the weights of a chunk.
"""
import pytest
import torch

import attention_attn_varlen_gb300 as av

DECAYS = (-0.0005, -0.01, -0.1, -1.0)
CUT_DECAY = -0.0007


def _exponential(x):
    return 2.0 ** -22 + x.abs() * 2.0 ** -24


def _tolerance(steps, g, segments):
    """Relative error allowed of e^(steps g), steps a tensor of token counts."""
    x64, near = (64 * g).abs(), (64 * g).abs() < 0.3
    chunk = 2.0 ** -24 + torch.where(near, 2.0 ** -23 * x64, _exponential(x64))
    tol = _exponential(steps.clamp(max=64) * g) + 2.0 ** -23 + torch.ceil(steps / 64) * chunk
    return tol + segments * (_exponential(steps * g / max(segments, 1)) + 2.0 ** -23)


def _cut_tolerance(steps, g):
    """The same in a sequence cut into segments, of 512 tokens at least."""
    return torch.stack([_tolerance(x, g, int(torch.ceil(x / 512))) for x in steps])


def _parts(w, n):
    """w (fp32) as the sum of n bf16 parts, in 64 bits."""
    left, total = w.double(), 0.0
    for _ in range(n):
        part = left.float().to(torch.bfloat16).double()
        total, left = total + part, left - part
    return total


def test_the_tolerance_tells_three_parts_from_two():
    for g in DECAYS[:3]:                                 # (e^-m of whole m: 64 weights only, most of them tiny)
        steps = torch.arange(1, 64, dtype=torch.float64)
        exact = torch.exp(steps * torch.tensor(g).double())
        tol = _tolerance(steps, torch.tensor(g).double(), 0) * exact
        assert ((_parts(exact.float(), 3) - exact).abs() <= tol).all()
        assert ((_parts(exact.float(), 2) - exact).abs() > 2 * tol).any()
    # the segments' tests: a weight of its chunk, wherever the chunks begin
    g, steps = torch.tensor(CUT_DECAY).double(), _steps_before(64)
    for begin in range(64):
        w = torch.exp((steps + begin) % 64 * g).float()
        assert ((_parts(w, 2) / w.double() - 1).abs() > 2 * _cut_tolerance(steps, g)).any()


def _steps_before(D):
    """Steps from a token to the sequence's end that lie before its last 448 tokens, one for each of D."""
    return 450 + 4 * torch.arange(D, dtype=torch.float64)


def _one_token_each(T, H, steps):
    """v with one token per value dimension, so many steps before the end."""
    v = torch.zeros(T, H, len(steps), dtype=torch.bfloat16)
    v[T - 1 - steps.long(), :, torch.arange(len(steps))] = 1.0
    return v


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("T", [2, 63, 64, 65, 200, 512])
def test_the_weights_of_a_prompt_are_fp32(T, D):
    H = len(DECAYS)
    g = torch.tensor(DECAYS)
    steps = (torch.arange(D) * T // D).double()
    v = _one_token_each(T, H, steps)
    ones = torch.ones(T, H, D, dtype=torch.bfloat16, device="cuda")
    # 40 sequences side by side: no sequence is cut
    B = 40
    cu = torch.arange(B + 1, dtype=torch.int32, device="cuda") * T
    s = torch.full((B, H, D, D), float("nan"), device="cuda")
    av.linear_attn_varlen_fwd(ones.repeat(B, 1, 1), ones.repeat(B, 1, 1), v.cuda().repeat(B, 1, 1), g.cuda(), cu, T,
                              state_cache=s, state_slots=torch.arange(B, dtype=torch.int32, device="cuda"))
    assert torch.equal(s, s[:1].expand(B, H, D, D))
    for h in range(H):
        want = torch.exp(steps * g[h].double())[:, None]
        err = (s[0, h].double().cpu() - want).abs()
        assert (err <= _tolerance(steps, g[h].double(), 0)[:, None] * want + 1e-37).all(), DECAYS[h]
    assert av.get_last_device_error()[0] == 0


@pytest.mark.gpu
@pytest.mark.parametrize("T,D", [(3000, 128), (2500, 64), (2503, 128)])
def test_the_weights_of_a_sequence_cut_into_segments_are_fp32(T, D):
    g, steps = torch.tensor([CUT_DECAY]), _steps_before(D)
    v = _one_token_each(T, 1, steps)
    ones = torch.ones(T, 1, D, dtype=torch.bfloat16, device="cuda")
    s = torch.full((1, 1, D, D), float("nan"), device="cuda")
    zero = torch.zeros(1, dtype=torch.int32, device="cuda")
    av.linear_attn_varlen_fwd(ones, ones, v.cuda(), g.cuda(), torch.tensor([0, T], dtype=torch.int32, device="cuda"), T,
                              state_cache=s, state_slots=zero)
    want = torch.exp(steps * g.double())[:, None]
    err = (s[0, 0].double().cpu() - want).abs()
    tol = _cut_tolerance(steps, g[0].double())
    assert (err <= tol[:, None] * want).all(), (err / want / tol[:, None]).max()
    assert av.get_last_device_error()[0] == 0


def _rounded_exponents(n):
    """n decays near -1 / 8192 whose e^(64 g) is at least a quarter of an fp32 step off its fp32 value."""
    out, g = [], torch.tensor(-1.0 / 8192)
    while len(out) < n:
        g = g * 1.003
        exact = torch.exp(64 * g.double())
        if abs(float(exact.float().double() - exact)) >= 2.0 ** -26:
            out.append(float(g))
    return torch.tensor(out)


@pytest.mark.gpu
def test_a_slow_decay_over_many_chunks_does_not_drift():
    """A large cached state and 8,192 tokens of zeros: e^(8192 g) times the state.  Each
    product's rounding goes either way and the mean over 4,096 entries loses it; what
    e^(64 g) is off by adds up over 128 chunks (2^-19 without its low part)."""
    H, D, T, B = 16, 64, 8192, 8                         # enough sequences and heads that none is cut
    g = _rounded_exponents(H)
    gen = torch.Generator(device="cuda").manual_seed(11)
    start = torch.randn(B, H, D, D, generator=gen, device="cuda") * 1000
    s, z = start.clone(), torch.zeros(B * T, H, D, dtype=torch.bfloat16, device="cuda")
    slots = torch.arange(B, dtype=torch.int32, device="cuda")
    out = av.linear_attn_varlen_fwd(z, z, z, g.cuda(), torch.arange(B + 1, dtype=torch.int32, device="cuda") * T, T,
                                    state_cache=s, state_slots=slots, context_lens=torch.ones_like(slots))
    assert out.eq(0).all()
    ratio = s.double() / (start.double() * torch.exp(T * g.double().cuda())[None, :, None, None])
    # 128 chunks of 2^-23 of 64 g (1 / 128 and a little), and roundings of 2^-24 each that do not add up
    assert (ratio.mean((0, 2, 3)) - 1).abs().max() <= 2.0 ** -22
    assert (ratio - 1).abs().max() <= 128 * 2.0 ** -24 + 2.0 ** -22
