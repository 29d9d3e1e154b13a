"""Sequences of the gated delta rule that are cut into segments, where something is out of
the ordinary: non-finite values in the first, a middle and the last segment, decays
and strengths at the ends of their range, sequences that start from zero, keep nothing or were refused,
slots out of range, offsets that ask for more segments than there is room for.

Tolerances: those of the other tests of the rule.  A segment's start is a product of its
predecessors' matrices with the first state; the steps' allowance covers its sums of D
terms (see test_long_sequences_cut_into_segments)."""
import functools

import pytest
import torch

import attention_attn_varlen_gb300 as av
from _delta_reference import delta
from _step_reference import cu_of
from test_gpu_delta_attn import check_out, check_state, i32, inputs

pytestmark = pytest.mark.gpu

T = 2900                                 # segments of 512 tokens
INF = float("inf")


def _is_cut(lens, Hk, Hv, D):
    assert av.delta_attn_workspace_size(len(lens), sum(lens), Hk, Hv, D, max(lens)) > 1 << 20


@functools.lru_cache(maxsize=None)
def _clean(H, D):
    host, _, gen = inputs(H + D, T, H, H, D)
    start = torch.randn(H, D, D, generator=gen)
    return start, delta(*host, [0, T], D ** -0.5, [start.double()], 1e-6)


@pytest.mark.parametrize("at", [0, 100, 511, 512, 1400, 2559, 2560, 2899])
@pytest.mark.parametrize("H,D", [(1, 128), (2, 64)])
def test_a_non_finite_value_in_a_segment(H, D, at):
    """One in v reaches its value dimension from its token on, over all later segments; one in k or beta everything
    of its head from its token on; one in q its own token's outputs."""
    _is_cut([T], H, H, D)
    start, (ref, finals, (rm, re)) = _clean(H, D)
    h = H - 1
    for which in ("v", "inf", "k", "q", "beta"):
        _, dev, _ = inputs(H + D, T, H, H, D)
        i = {"q": 0, "k": 1, "v": 2, "inf": 2, "beta": 4}[which]
        bad = INF if which == "inf" else float("nan")
        if which == "beta":
            dev[i][at, h] = bad
        else:
            dev[i][at, h, 5] = bad
        s = start[None].cuda()
        out = av.delta_attn_varlen_fwd(*dev, i32(0, T), T, state_cache=s, state_slots=i32(0), context_lens=i32(1),
                                       qk_norm_eps=1e-6)
        hit = torch.zeros(T, H, D, dtype=torch.bool)
        if which == "q":
            hit[at, h] = True
        elif i == 2:
            hit[at:, h, 5] = True
        else:
            hit[at:, h] = True
        got = out.cpu()
        assert not torch.isfinite(got[hit].float()).any(), which
        check_out(got[~hit], ref[~hit], (rm[~hit], re[~hit]), which)
        got, rows = s[0].cpu(), hit[-1] if which != "q" else torch.zeros(H, D, dtype=torch.bool)
        assert not torch.isfinite(got[rows]).any(), which
        S, E = finals[0]
        check_state(got[~rows], S[~rows], E[~rows], which)
    assert av.get_last_device_error()[0] == 0


@pytest.mark.parametrize("D", [64, 128])
def test_decays_and_strengths_at_the_ends_over_segments(D):
    H = 4
    _is_cut([T], H, H, D)
    host, dev, _ = inputs(6, T, H, H, D)
    for x, y in (host[3:], dev[3:]):
        x[:, 0], x[:, 1], x[:, 2] = 0.0, -1e-4, -40.0
        x[::500, 3] = -INF                                   # among them whole segments without one
        x[1000:1100, 3] = -300.0
        y[:, 0], y[:, 1] = 1.0, 0.5
        y[10:2000:2, 2], y[60:1200, 3] = 0.0, 0.0            # a segment that writes nothing
    sd = torch.full((1, H, D, D), float("nan"), device="cuda")          # never read
    out = av.delta_attn_varlen_fwd(*dev, i32(0, T), T, 1.0, state_cache=sd, state_slots=i32(0), qk_norm_eps=0.0)
    ref, finals, reach = delta(*host, [0, T], 1.0, [None], 0.0)
    check_out(out, ref, reach, "out")
    check_state(sd[0], *finals[0], "state")
    assert av.get_last_device_error()[0] == 0


@pytest.mark.parametrize("H,D", [(1, 128), (2, 64)])
def test_starts_slots_and_refusals_of_cut_sequences(H, D):
    lens = [2600, 30, 1800, 0, 2300]
    B, total, cu = len(lens), sum(lens), cu_of(lens)
    _is_cut(lens, H, H, D)
    host, dev, gen = inputs(17, total, H, H, D)
    state = torch.randn(6, H, D, D, generator=gen)
    zero, _, zero_reach = delta(*host, cu, D ** -0.5, [None] * B, 1e-6)
    for name, slots, past, grown, error in (
            ("zero starts", [4, 0, 2, 1, 3], [0, 0, 0, 0, 0], None, 0),
            ("nothing kept", [-1, 5, -1, 1, -1], [9, 9, 9, 9, 9], None, 0),
            ("some refused", [4, 0, 2, 1, 3], [9, 9, 0, 9, 9], [9, 9 + 30, 0, 9, 9 + 2300], 0),
            ("out of range", [6, 0, 1 << 30, 1, 3], [9, 0, 9, 9, 9], None, 6)):
        sd = state.clone()
        kept = [b for b in range(B) if 0 <= slots[b] < 6 and not (grown and grown[b] <= past[b])]
        for b in kept:
            if past[b] == 0 and lens[b]:
                sd[slots[b]] = float("nan")                  # never read
        before, sd = sd.clone(), sd.cuda()
        av.get_last_device_error()
        out = av.delta_attn_varlen_fwd(*dev, cu.cuda(), max(lens), state_cache=sd, state_slots=i32(*slots),
                                       context_lens=i32(*past), cache_seqlens=i32(*grown) if grown else None,
                                       qk_norm_eps=1e-6)
        assert av.get_last_device_error()[0] == error, name
        starts = [before[slots[b]].double() if b in kept and past[b] else None for b in range(B)]
        if any(x is not None for x in starts):
            ref, finals, reach = delta(*host, cu, D ** -0.5, starts, 1e-6)
        else:
            ref, finals, reach = zero, None, zero_reach
        check_out(out, ref, reach, name)
        got, changed = sd.cpu(), [slots[b] for b in kept if lens[b]]
        if finals is None:
            finals = delta(*host, cu, D ** -0.5, starts, 1e-6)[1]
        for b in kept:
            if lens[b]:
                check_state(got[slots[b]], *finals[b], f"{name} {b}")
        rest = [x for x in range(6) if x not in changed]
        assert torch.equal(got[rest], before[rest]), name
    # without a cache, and padded behind the last sequence
    more = [torch.cat([x, torch.full_like(x[:70], float("nan"))]) for x in dev]
    out = torch.full((total + 70, H, D), 7.0, dtype=torch.bfloat16, device="cuda")
    av.delta_attn_varlen_fwd(*more, cu.cuda(), max(lens), out=out, qk_norm_eps=1e-6)
    check_out(out[:total], zero, zero_reach, "no cache")
    assert out[total:].eq(7.0).all() and av.get_last_device_error()[0] == 0


@pytest.mark.parametrize("lens,Hk,Hv,D", [([1] * 7, 1, 2, 64), ([2, 5, 8], 2, 2, 128), ([9, 16, 12], 1, 2, 64),
                                          ([40, 200, 64], 2, 2, 128), ([300, 31], 1, 4, 64), ([T], 1, 1, 128),
                                          ([T], 1, 2, 64)])
@pytest.mark.parametrize("same", [False, True])
def test_strengths_between_one_and_two(lens, Hk, Hv, D, same):
    """beta in [1, 2] turns a state around along a key; same: one key again and again, in
    whose direction the inverse's entries reach 2.  (I - beta k k^T) still lengthens nothing, so the reach is the
    same recursion; the inverse's entries are at most beta, and the writes twice as long
    against it: twice the allowances."""
    B, total = len(lens), sum(lens)
    host, dev, gen = inputs(total + D, total, Hk, Hv, D)
    beta = 1 + torch.rand(total, Hv, generator=gen)
    beta[::3, 0], beta[1::5, -1] = 2.0, 1.0
    g = host[3] * 0.05
    if same:
        for x in (host, dev):
            x[1][:] = x[1][0].clone()
    host, dev = (*host[:3], g, beta), (*dev[:3], g.cuda(), beta.cuda())
    state = torch.randn(B, Hv, D, D, generator=gen)
    sd, slots, past = state.cuda(), i32(*range(B)), i32(*[3] * B)
    av.get_last_device_error()
    kw = dict(state_cache=sd, state_slots=slots, context_lens=past, qk_norm_eps=1e-6)
    out = av.delta_attn_varlen_fwd(*dev, cu_of(lens).cuda(), max(lens), **kw)
    ref, finals, (rm, re) = delta(*host, cu_of(lens), D ** -0.5, list(state.double()), 1e-6)
    check_out(out, ref, (2 * rm, 2 * re), "out")
    for b in range(B):
        S, E = finals[b]
        check_state(sd[b], S, 2 * E, str(b))
    if max(lens) == 1:
        sd.copy_(state)
        again = av.delta_attn_decode(*dev, sd, slots, context_lens=past, qk_norm_eps=1e-6)
        check_out(again, ref, (2 * rm, 2 * re), "decode")
    assert av.get_last_device_error()[0] == 0


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("tokens", [2900, 2560])
@pytest.mark.parametrize("n", [20, 40, 101])
def test_more_segments_than_there_is_room_for(D, tokens, n):
    """Offsets that go back and forth, so that n sequences share the same tokens, the last of their
    segments shorter or not: reported.  States are the right ones or untouched and no output is
    a wrong one, whatever the workspace held; what is not a sequence's is not written."""
    H = 1
    host, dev, gen = inputs(3, tokens + 50, H, H, D)
    host = tuple(x[:tokens] for x in host)
    cu = i32(*([0, tokens] * n))
    B = 2 * n - 1
    state = torch.randn(B + 1, H, D, D, generator=gen)
    sd = state.cuda()
    out = torch.full((tokens + 50, H, D), 7.0, dtype=torch.bfloat16, device="cuda")
    ws = torch.full((av.delta_attn_workspace_size(B, tokens + 50, H, H, D, tokens),), 0xFF, dtype=torch.uint8,
                    device="cuda")                           # NaN
    assert ws.numel() > 1 << 20
    av.get_last_device_error()
    av.delta_attn_varlen_fwd(*dev, cu, tokens, state_cache=sd,
                             state_slots=torch.arange(B, dtype=torch.int32, device="cuda"), out=out, workspace=ws,
                             qk_norm_eps=1e-6)
    assert av.get_last_device_error()[0] == 6
    got, (ref, finals, reach) = sd.cpu(), delta(*host, [0, tokens], D ** -0.5, [None], 1e-6)
    assert out[tokens:].eq(7.0).all()
    written = ~out[:tokens].eq(7.0).all(-1).all(-1).cpu()
    assert written[:512].all()
    check_out(out[:tokens][written.cuda()], ref[written], tuple(x[written] for x in reach), "out")
    assert torch.equal(got[1::2], state[1::2])               # the backward ones are no sequences
    run = [b for b in range(0, B, 2) if not torch.equal(got[b], state[b])]
    for b in run:
        check_state(got[b], *finals[0], str(b))
    # room for 2 n - 1 + 153 units; those of the shorter last segments lie behind all others
    segments = -(-tokens // 512)
    room = 2 * n - 1 + 153 - segments * n
    assert len(run) == (n if room >= 0 else max(0, n + room) if tokens % 512 else len(run))
    # the next call is an ordinary one
    s = torch.zeros(1, H, D, D, device="cuda")
    av.delta_attn_varlen_fwd(*dev, i32(0, tokens), tokens, state_cache=s, state_slots=i32(0), qk_norm_eps=1e-6)
    check_state(s[0], *finals[0], "after")
    assert av.get_last_device_error()[0] == 0
