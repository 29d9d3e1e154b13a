"""linear_attn_varlen_fwd / linear_attn_decode on the GPU against the recurrence
in 64 bits, token after token.

Tolerances.  An output is rounded once to bf16 (2^-8 of it); the fp32 sums and
the terms' own errors are bounded by the sum of the terms' absolute values
(`weight`): terms carried as two bf16 parts are off by at most 2^-16 each, one
such factor per product, exponentials by 2^-20, and fp32 sums of up to 4096
terms by 2^-12 * 2^-4 at the very worst; 2^-14 of the weight covers them.  A
state is fp32: terms carried as three bf16 parts (2^-24), e^(n g) of up to a
chunk's length (2^-21) and fp32 sums: 2^-17 of the sum of absolute values.  A
state that advances in steps (tokens, or fewer where they are taken together)
multiplies e^g's own rounding and its sum's with every step: 2^-23 of the weight
for each token of the sequence, in the state and in what is read from it.
"""
import pytest
import torch

import attention_attn_varlen_gb300 as av
from _step_reference import cu_of, linear

pytestmark = pytest.mark.gpu


def _check(got, ref, weight, what):
    err = (got.double().cpu() - ref).abs()
    tol = 2.0 ** -8 * ref.abs() + (2.0 ** -14 + len(ref) * 2.0 ** -23) * weight
    assert torch.isfinite(got.float()).all(), what
    assert (err <= tol).all(), f"{what}: worst {(err / tol.clamp(min=1e-30)).max():.2f} of the tolerance"
    rel = (err.norm() / ref.norm().clamp(min=1e-30)).item()
    assert rel <= 2.5e-3, f"{what}: relative error {rel:.2e}"      # a rounding to bf16 alone: 1.7e-3


def _check_state(got, ref, weight, what, steps=1000):
    err = (got.double().cpu() - ref).abs()
    assert (err <= (2.0 ** -17 + steps * 2.0 ** -23) * weight + 1e-30).all(), f"{what}: {(err / weight.clamp(min=1e-30)).max():.2e} of the weight"


def _inputs(seed, T, Hq, Hkv, D, strided=True):
    gen = torch.Generator().manual_seed(seed)
    qkv = torch.randn(T, Hq + 2 * Hkv, D, generator=gen).to(torch.bfloat16)
    d = qkv.cuda()
    parts = lambda x: (x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:])  # noqa: E731
    dev = parts(d)
    if not strided:
        dev = tuple(x.contiguous() for x in dev)
    return parts(qkv), dev, gen


def _decay(Hkv):
    return (-(2.0 ** (-8.0 * torch.arange(1, Hkv + 1, dtype=torch.float64) / Hkv))).float()


@pytest.mark.parametrize("lens,Hq,Hkv,D,strided", [
    ([1], 1, 1, 64, True), ([1], 2, 2, 128, False), ([63, 64, 65], 2, 2, 128, True), ([1, 2, 0, 3, 130], 4, 2, 64, True),
    ([200, 0, 1, 77], 3, 1, 128, True), ([129, 300], 8, 2, 64, False), ([512], 4, 4, 128, True),
    ([17] * 20, 4, 4, 64, True), ([1000, 5], 2, 1, 128, True), ([640], 2, 2, 64, True)])
@pytest.mark.parametrize("cached", [False, True])
def test_prompts_match_the_recurrence(lens, Hq, Hkv, D, strided, cached):
    B, T = len(lens), sum(lens)
    (q, k, v), dev, gen = _inputs(T + D, T, Hq, Hkv, D, strided)
    g, cu, scale = _decay(Hkv), cu_of(lens), D ** -0.5
    state = torch.randn(B + 2, Hkv, D, D, generator=gen)
    slots = torch.randperm(B + 2, generator=gen)[:B].to(torch.int32)
    ctx = torch.tensor([b % 2 * 10 for b in range(B)], dtype=torch.int32)
    sd = state.cuda()
    av.get_last_device_error()
    kw = dict(state_cache=sd, state_slots=slots.cuda(), context_lens=ctx.cuda()) if cached else {}
    out = av.linear_attn_varlen_fwd(*dev, g.cuda(), cu.cuda(), max(lens), scale, **kw)
    torch.cuda.synchronize()
    assert av.get_last_device_error()[0] == 0
    starts = [state[slots[b]].double() if cached and ctx[b] > 0 else None for b in range(B)]
    ref, finals, weight = linear(q, k, v, g, cu, scale, starts)
    _check(out, ref, weight, "out")
    if cached:
        got = sd.cpu()
        for b in range(B):
            if lens[b] == 0:
                assert torch.equal(got[slots[b]], state[slots[b]])
            else:
                _check_state(got[slots[b]], *finals[b], f"state {b}", lens[b])
        free = [s for s in range(B + 2) if s not in slots.tolist()]
        assert torch.equal(got[free], state[free])


@pytest.mark.parametrize("B,Hq,Hkv,D,strided", [(1, 1, 1, 64, True), (3, 8, 2, 128, True), (40, 4, 4, 64, False),
                                                (7, 5, 1, 128, True), (130, 2, 2, 128, False)])
def test_decode_matches_the_recurrence(B, Hq, Hkv, D, strided):
    (q, k, v), dev, gen = _inputs(B + D, B, Hq, Hkv, D, strided)
    g, scale = _decay(Hkv), 0.3
    state = torch.randn(B + 2, Hkv, D, D, generator=gen)
    slots = torch.randperm(B + 2, generator=gen)[:B].to(torch.int32)
    if B > 2:
        slots[1] = -1
    ctx = torch.ones(B, dtype=torch.int32)
    ctx[::3] = 0
    for use_ctx in (False, True):
        sd = state.cuda()
        av.get_last_device_error()
        out = av.linear_attn_decode(*dev, g.cuda(), sd, slots.cuda(), scale, context_lens=ctx.cuda() if use_ctx else None)
        torch.cuda.synchronize()
        assert av.get_last_device_error()[0] == 0
        starts = [state[slots[b]].double() if slots[b] >= 0 and not (use_ctx and ctx[b] == 0) else None
                  for b in range(B)]
        ref, finals, weight = linear(q, k, v, g, list(range(B + 1)), scale, starts)
        _check(out, ref, weight, "out")
        got, want = sd.cpu(), state.clone()
        for b in range(B):
            if slots[b] >= 0:
                _check_state(got[slots[b]], *finals[b], f"state {b}", 1)
                want[slots[b]] = got[slots[b]]
        assert torch.equal(got, want)


@pytest.mark.parametrize("D", [64, 128])
def test_decays_at_the_ends_of_their_range(D):
    """No decay, a slow one over many chunks, one that is gone after a token, and
    e^g = 0 (only the token itself)."""
    g = torch.tensor([0.0, -1e-4, -40.0, float("-inf")])
    lens = [700, 3]
    (q, k, v), dev, _ = _inputs(5, 703, 4, 4, D)
    sd = torch.full((2, 4, D, D), float("nan"), device="cuda")          # never read: both start from zero
    av.get_last_device_error()
    out = av.linear_attn_varlen_fwd(*dev, g.cuda(), cu_of(lens).cuda(), 700, 1.0, state_cache=sd,
                                    state_slots=torch.tensor([1, 0], dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    assert av.get_last_device_error()[0] == 0
    ref, finals, weight = linear(q, k, v, g, cu_of(lens), 1.0, [None, None])
    _check(out, ref, weight, "out")
    _check_state(sd[1], *finals[0], "state")
    _check_state(sd[0], *finals[1], "state")


def test_the_tokens_of_a_prompt_one_by_one_and_in_pieces_agree():
    """A prompt at once, in uneven pieces that continue from the cached state, and
    token by token through the recurrent form."""
    T, H, D = 150, 2, 128
    (q, k, v), (qd, kd, vd), _ = _inputs(9, T, H, H, D)
    g = _decay(H).cuda()
    ref, finals, weight = linear(q, k, v, g.cpu(), [0, T], D ** -0.5, [None])
    slot = torch.zeros(1, dtype=torch.int32, device="cuda")
    for pieces in ([150], [1, 64, 20, 65], [149, 1], [1] * 150):
        s = torch.full((1, H, D, D), float("nan"), device="cuda")
        out, at = [], 0
        for n in pieces:
            past = torch.tensor([at], dtype=torch.int32, device="cuda")
            x = (qd[at:at + n], kd[at:at + n], vd[at:at + n])
            if len(pieces) == T:
                out.append(av.linear_attn_decode(*x, g, s, slot, context_lens=past))
            else:
                out.append(av.linear_attn_varlen_fwd(*x, g, cu_of([n]).cuda(), n, state_cache=s, state_slots=slot,
                                                     context_lens=past))
            at += n
        _check(torch.cat(out), ref, weight, str(len(pieces)))
        _check_state(s[0], *finals[0], str(len(pieces)))


@pytest.mark.parametrize("D", [64, 128])
def test_rows_of_other_sequences_and_behind_the_last_do_not_reach_a_sequence(D):
    """NaN and infinities in another sequence, in rows behind the last one and in
    unused state slots: outputs and states of a sequence do not see them, and rows
    behind the last sequence are left as they were."""
    lens, H = [70, 33, 5], 2
    T = sum(lens)
    (q, k, v), dev, _ = _inputs(3, T + 80, H, H, D, strided=False)
    for x in dev:
        x[70:103] = float("nan")
        x[70::2, :, ::3] = float("inf")
        x[103:108] = 1.0
        x[108:] = float("nan")
    for x in (q, k, v):
        x[103:108] = 1.0
    out = torch.full((T + 80, H, D), 7.0, dtype=torch.bfloat16, device="cuda")
    sd = torch.full((5, H, D, D), float("nan"), device="cuda")
    slots = torch.tensor([4, -1, 0], dtype=torch.int32, device="cuda")
    g = _decay(H)
    av.linear_attn_varlen_fwd(*dev, g.cuda(), cu_of(lens).cuda(), 70, 1.0, state_cache=sd, state_slots=slots, out=out)
    torch.cuda.synchronize()
    for b, a, e in ((0, 0, 70), (2, 103, 108)):
        ref, finals, weight = linear(q[a:e], k[a:e], v[a:e], g, [0, e - a], 1.0, [None])
        _check(out[a:e], ref, weight, f"sequence {b}")
        _check_state(sd[slots[b]], *finals[0], f"state {b}")
    assert out[T:].eq(7.0).all()
    assert sd[1:4].isnan().all()


def test_bad_indices_are_reported_and_skipped():
    D, H = 64, 2
    _, dev, _ = _inputs(4, 20, H, H, D)
    g = _decay(H).cuda()
    sd = torch.zeros(2, H, D, D, device="cuda")
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    av.get_last_device_error()
    # offsets past the tokens, decreasing offsets
    out = torch.full((20, H, D), 7.0, dtype=torch.bfloat16, device="cuda")
    av.linear_attn_varlen_fwd(*dev, g, i32(0, 10, 5, 90), 20, state_cache=sd, state_slots=i32(0, 1, 1), out=out)
    assert av.get_last_device_error()[0] == 6
    assert out[10:].eq(7.0).all() and not out[:10].eq(7.0).all() and sd[1].eq(0).all()
    # a slot past the cache: the sequence runs from zero and keeps nothing
    a = av.linear_attn_varlen_fwd(*dev, g, i32(0, 20), 20, state_cache=sd, state_slots=i32(2), context_lens=i32(5))
    assert av.get_last_device_error()[0] == 6
    b = av.linear_attn_varlen_fwd(*dev, g, i32(0, 20), 20)
    assert torch.equal(a, b)
    av.linear_attn_decode(dev[0][:1], dev[1][:1], dev[2][:1], g, sd, i32(7))
    assert av.get_last_device_error()[0] == 6
    # longer than max_seqlen: cut and reported
    out.fill_(7.0)
    av.linear_attn_varlen_fwd(*dev, g, i32(0, 20), 12, out=out)
    assert av.get_last_device_error()[0] == 6
    assert torch.equal(out[:12], b[:12]) and out[12:].eq(7.0).all()
    # a positive and a NaN decay count as none
    bad = torch.tensor([0.5, float("nan")], device="cuda")
    c = av.linear_attn_varlen_fwd(*dev, bad, i32(0, 20), 20)
    assert av.get_last_device_error()[0] == 8
    assert torch.equal(c, av.linear_attn_varlen_fwd(*dev, torch.zeros(2, device="cuda"), i32(0, 20), 20))
    assert av.get_last_device_error()[0] == 0


def test_repeated_calls_and_other_streams_give_the_same_bits():
    lens = [333, 64, 1]
    _, dev, gen = _inputs(12, sum(lens), 4, 2, 128)
    g, cu = _decay(2).cuda(), cu_of(lens).cuda()
    state = torch.randn(3, 2, 128, 128, generator=gen).cuda()
    slots, ctx = torch.arange(3, dtype=torch.int32, device="cuda"), torch.ones(3, dtype=torch.int32, device="cuda")

    def call(stream=None):
        s = state.clone()
        torch.cuda.synchronize()
        o = av.linear_attn_varlen_fwd(*dev, g, cu, 333, state_cache=s, state_slots=slots, context_lens=ctx,
                                      stream=stream)
        torch.cuda.synchronize()
        return o, s

    o, s = call()
    for stream in (None, torch.cuda.Stream()):
        o2, s2 = call(stream)
        assert torch.equal(o, o2) and torch.equal(s, s2)


def test_captured_decode_steps_advance_the_state():
    B, H, D = 4, 2, 128
    (q, k, v), dev, _ = _inputs(31, 5 * B, H, H, D, strided=False)
    g = _decay(H)
    sd = torch.zeros(B, H, D, D, device="cuda")
    slots = torch.arange(B, dtype=torch.int32, device="cuda")
    x = [t[:B].clone() for t in dev]
    out = torch.empty_like(x[0])
    av.linear_attn_decode(*x, g.cuda(), sd, slots, out=out)
    graph, gd = torch.cuda.CUDAGraph(), g.cuda()
    with torch.cuda.graph(graph):
        av.linear_attn_decode(*x, gd, sd, slots, out=out)
    for step in range(1, 5):
        for a, b in zip(x, dev):
            a.copy_(b[step * B:(step + 1) * B])
        graph.replay()
    torch.cuda.synchronize()
    order = [step * B + b for b in range(B) for step in range(5)]
    ref, finals, weight = linear(q[order], k[order], v[order], g, [5 * b for b in range(B + 1)], D ** -0.5, [None] * B)
    _check(out, ref[4::5], weight[4::5], "last step")
    for b in range(B):
        _check_state(sd[b], *finals[b], f"state {b}")


def test_no_tokens_leaves_the_states():
    q = torch.empty(0, 2, 64, dtype=torch.bfloat16, device="cuda")
    sd = torch.ones(2, 2, 64, 64, device="cuda")
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    out = av.linear_attn_varlen_fwd(q, q, q, _decay(2).cuda(), i32(0, 0, 0), 0, state_cache=sd, state_slots=i32(0, 1))
    assert out.shape == q.shape and sd.eq(1).all() and av.get_last_device_error()[0] == 0


@pytest.mark.parametrize("lens,Hq,Hkv,D", [([2500, 70], 2, 1, 64), ([3000], 2, 2, 128), ([1, 1900, 0, 2300], 3, 3, 64)])
@pytest.mark.parametrize("cached", [False, True])
def test_long_sequences_cut_into_segments(lens, Hq, Hkv, D, cached):
    """Few heads and long sequences: segments side by side, from states that a first
    pass over k and v prepares."""
    B, T = len(lens), sum(lens)
    (q, k, v), dev, gen = _inputs(T, T, Hq, Hkv, D)
    g, cu = torch.tensor([-0.002, -0.2, 0.0])[:Hkv], cu_of(lens)
    state = torch.randn(B, Hkv, D, D, generator=gen)
    ctx = torch.ones(B, dtype=torch.int32) if cached else torch.zeros(B, dtype=torch.int32)
    sd = state.cuda()
    av.get_last_device_error()
    out = av.linear_attn_varlen_fwd(*dev, g.cuda(), cu.cuda(), max(lens), 0.1, state_cache=sd,
                                    state_slots=torch.arange(B, dtype=torch.int32, device="cuda"),
                                    context_lens=ctx.cuda())
    torch.cuda.synchronize()
    assert av.get_last_device_error()[0] == 0
    ref, finals, weight = linear(q, k, v, g, cu, 0.1, [state[b].double() if cached else None for b in range(B)])
    _check(out, ref, weight, "out")
    for b in range(B):
        if lens[b]:
            _check_state(sd[b], *finals[b], f"state {b}", lens[b])


@pytest.mark.parametrize("D,bad", [(64, float("nan")), (128, float("inf")), (128, float("nan"))])
def test_a_non_finite_value_reaches_its_own_token_and_later_ones_only(D, bad):
    """One entry of v, k or q: other value dimensions, heads and the earlier tokens,
    those of the same chunk among them, are what they are without it."""
    T, H, t, d = 200, 2, 101, 37
    _, dev, _ = _inputs(77, T, H, H, D, strided=False)
    g, cu = _decay(H).cuda(), cu_of([T]).cuda()
    clean = av.linear_attn_varlen_fwd(*dev, g, cu, T)
    for which in range(3):
        x = [y.clone() for y in dev]
        x[which][t, 1, d] = bad
        out = av.linear_attn_varlen_fwd(*x, g, cu, T)
        assert torch.equal(out[:t], clean[:t]) and torch.equal(out[:, 0], clean[:, 0])
        if which == 2:      # v: one value dimension, from its token on
            others = [i for i in range(D) if i != d]
            assert torch.equal(out[:, 1][:, others], clean[:, 1][:, others])
            assert not out[t:, 1, d].isfinite().any()
        elif which == 1:    # k: the whole head from its token on
            assert not out[t:, 1].isfinite().any()
        else:               # q: its own token
            assert not out[t, 1].isfinite().any() and torch.equal(out[t + 1:], clean[t + 1:])


@pytest.mark.parametrize("Hq,Hkv,D", [(16, 4, 128), (12, 12, 64)])
def test_many_sequences_give_the_bits_of_each_alone(Hq, Hkv, D):
    """Far more (sequence, head) pairs than the GPU has SMs, of mixed lengths: each
    one's output and state are those of a call with it alone, and NaN and infinities
    of one do not reach what is computed after it."""
    lens = [(7 * i * i + 13 * i) % 400 for i in range(50)] + [64, 128, 1, 1, 0, 63, 65]
    B, T = len(lens), sum(lens)
    _, dev, gen = _inputs(Hq + D, T, Hq, Hkv, D)
    cu, g = cu_of(lens), _decay(Hkv).cuda()
    bad = [b for b in range(B) if b % 5 == 2 and lens[b]]
    for b in bad:
        for i, x in enumerate(dev):
            x[int(cu[b]) + lens[b] // 2, 0, i] = float("inf") if b % 2 else float("nan")
    state = torch.randn(B, Hkv, D, D, generator=gen).cuda()
    slots = torch.randperm(B, generator=gen).to(torch.int32).cuda()
    ctx = torch.tensor([b % 3 for b in range(B)], dtype=torch.int32, device="cuda")
    sd = state.clone()
    out = av.linear_attn_varlen_fwd(*dev, g, cu.cuda(), max(lens), state_cache=sd, state_slots=slots, context_lens=ctx)
    assert av.get_last_device_error()[0] == 0
    same = lambda a, b: torch.equal(a.view(torch.int16), b.view(torch.int16))  # noqa: E731
    for b in range(B):
        a, e = int(cu[b]), int(cu[b + 1])
        s1, at = state.clone(), int(slots[b])
        one = av.linear_attn_varlen_fwd(*(x[a:e] for x in dev), g, cu_of([e - a]).cuda(), max(lens), state_cache=s1,
                                        state_slots=slots[b:b + 1], context_lens=ctx[b:b + 1])
        assert b in bad or (one.isfinite().all() and s1[at].isfinite().all())
        assert same(out[a:e], one) if b not in bad else torch.equal(out[a:e].isnan(), one.isnan())
        assert same(sd[at], s1[at]) if b not in bad else torch.equal(sd[at].isfinite(), s1[at].isfinite())
    assert av.get_last_device_error()[0] == 0


def test_captured_prompts_replay_on_new_lengths_and_share_a_workspace():
    """Two graphs over one workspace, replayed in turn with other tokens and other
    lengths within max_seqlen."""
    B, T, Hq, Hkv, D, most = 5, 900, 4, 2, 128, 700
    _, dev, _ = _inputs(8, T, Hq, Hkv, D, strided=False)
    g = _decay(Hkv).cuda()
    ws = torch.empty(av.linear_attn_workspace_size(B, Hq, Hkv, D, most), dtype=torch.uint8, device="cuda")
    slots, ctx = torch.arange(B, dtype=torch.int32, device="cuda"), torch.ones(B, dtype=torch.int32, device="cuda")
    graphs = []
    for i in range(2):
        x, cu = [t.clone() for t in dev], torch.zeros(B + 1, dtype=torch.int32, device="cuda")
        sd, out = torch.zeros(B, Hkv, D, D, device="cuda"), torch.zeros(T, Hq, D, dtype=torch.bfloat16, device="cuda")
        call = lambda: av.linear_attn_varlen_fwd(*x, g, cu, most, state_cache=sd, state_slots=slots,  # noqa: E731
                                                 context_lens=ctx, out=out, workspace=ws)
        call()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call()
        graphs.append((graph, x, cu, sd, out))
    steps = [[10, 0, 64, 65, 700], [1, 1, 1, 1, 1], [300, 300, 300, 0, 0], [0, 0, 0, 0, 129]]
    want = [torch.zeros(B, Hkv, D, D, device="cuda") for _ in graphs]
    for n, lens in enumerate(steps):
        for i, (graph, x, cu, sd, out) in enumerate(graphs):
            for t, src in zip(x, dev):
                t.copy_(src.roll(n + 3 * i, 0))
            cu.copy_(cu_of(lens))
            graph.replay()
            got = out[:sum(lens)].clone()
            ref = av.linear_attn_varlen_fwd(*x, g, cu, most, state_cache=want[i], state_slots=slots, context_lens=ctx)
            assert torch.equal(got, ref[:sum(lens)]) and torch.equal(sd, want[i])
    assert av.get_last_device_error()[0] == 0


def test_states_and_rows_past_32_bits_of_offset():
    """A state slot and rows further than 2^31 elements from the first."""
    Hq, Hkv, D, num = 8, 8, 128, 16400                    # 2^17 elements a slot
    (q, k, v), dev, gen = _inputs(2, 70, Hq, Hkv, D)
    g, i32 = _decay(Hkv), lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    sd = torch.empty(num, Hkv, D, D, device="cuda")
    start = torch.randn(Hkv, D, D, generator=gen)
    sd[num - 1] = start.cuda()
    stride = 1 << 25                                      # row 64 is 2^31 elements behind row 0
    far = [torch.empty(70 * stride, dtype=torch.bfloat16, device="cuda").as_strided((70, Hq, D), (stride, D, 1))
           for _ in range(2)]
    far[0].copy_(dev[0])
    out = av.linear_attn_varlen_fwd(far[0], *dev[1:], g.cuda(), i32(0, 70), 70, state_cache=sd, state_slots=i32(num - 1),
                                    context_lens=i32(1), out=far[1])
    ref, finals, weight = linear(q, k, v, g, [0, 70], D ** -0.5, [start.double()])
    _check(out, ref, weight, "out")
    _check_state(sd[num - 1], *finals[0], "state")
    sd[num - 1] = start.cuda()
    out = av.linear_attn_decode(far[0][65:66], *(x[65:66] for x in dev[1:]), g.cuda(), sd, i32(num - 1), out=far[1][66:67])
    ref, finals, weight = linear(q[65:66], k[65:66], v[65:66], g, [0, 1], D ** -0.5, [start.double()])
    _check(out, ref, weight, "out")
    _check_state(sd[num - 1], *finals[0], "state", 1)
    assert av.get_last_device_error()[0] == 0


def test_the_largest_batch_and_a_wide_group():
    """65,535 sequences of one token or none; 48 query heads on one state."""
    B, D = 65535, 64
    gen = torch.Generator().manual_seed(4)
    lens = torch.randint(0, 2, (B,), generator=gen)
    T = int(lens.sum())
    q, k, v = (torch.randn(T, 1, D, generator=gen).to(torch.bfloat16) for _ in range(3))
    slots = torch.full((B,), -1, dtype=torch.int32)
    slots[::1000] = torch.arange(len(slots[::1000]), dtype=torch.int32)
    sd = torch.full((70, 1, D, D), 3.0, device="cuda")
    g = torch.tensor([-0.5], device="cuda")
    out = av.linear_attn_varlen_fwd(q.cuda(), k.cuda(), v.cuda(), g, cu_of(lens.tolist()).cuda(), 1, 0.5, state_cache=sd,
                                    state_slots=slots.cuda())
    qk = 0.5 * (q.double() * k.double()).sum(-1, keepdim=True)
    _check(out[:, 0], (qk * v.double())[:, 0], (0.5 * (q.double() * k.double()).abs().sum(-1, keepdim=True)
                                                * v.double().abs())[:, 0], "one token each")
    at = torch.cumsum(lens, 0) - 1
    for b in range(0, B, 1000):
        got = sd[slots[b], 0].double().cpu()
        want = torch.outer(v[at[b], 0].double(), k[at[b], 0].double()) if lens[b] else torch.full((D, D), 3.0).double()
        assert ((got - want).abs() <= 2.0 ** -22 * want.abs()).all()
    (q, k, v), dev, _ = _inputs(7, 100, 48, 1, 64)
    s1 = torch.randn(1, 1, 64, 64, generator=gen)
    sd = s1.cuda()
    zero, one = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.ones(1, dtype=torch.int32, device="cuda")
    out = av.linear_attn_varlen_fwd(*dev, g, cu_of([100]).cuda(), 100, state_cache=sd, state_slots=zero, context_lens=one)
    ref, finals, weight = linear(q, k, v, g.cpu(), [0, 100], 64 ** -0.5, [s1[0].double()])
    _check(out, ref, weight, "48 heads")
    _check_state(sd[0], *finals[0], "48 heads", 100)
    assert av.get_last_device_error()[0] == 0
