"""delta_attn_varlen_fwd / delta_attn_decode on the GPU against the recurrence in 64
bits, token after token.

Tolerances.  A step's own error, relative to M_t (the length a row of the state can
have, see _delta_reference.delta): the recurrent form sums S k and S q over a
lane's four terms and a tree of five, nine roundings, and makes some fifteen more for
the decay, the norms, u and the new state: 32 x 2^-24.  The chunked form carries every
operand as parts of 2^-24 together; the solve's rows add up to 64 terms bounded
by M (the inverse's entries are at most 1 for beta in [0, 1] and keys no longer than 1),
again in fp32: 128 x 2^-24 a step covers both.  Outputs are rounded once to bf16: half a
step of 2^-7, at most 2^-8 of them (8 significant bits: next to a power of two the step is
2^-7 of the value); the chunked form takes the state and q . k factors of an output as two
bf16 parts each: 2^-16 a factor, three factors, 2^-14 of scale |q| M.
"""
import functools

import pytest
import torch

import attention_attn_varlen_gb300 as av
from _delta_reference import delta
from _step_reference import cu_of

pytestmark = pytest.mark.gpu

STEP = 128 * 2.0 ** -24


def check_out(got, ref, reach, what):
    rm, re = reach
    err = (got.double().cpu() - ref).abs()
    tol = 2.0 ** -8 * ref.abs() + 2.0 ** -14 * rm + STEP * re + 1e-30
    assert torch.isfinite(got.float()).all(), what
    assert (err <= tol).all(), f"{what}: worst {(err / tol).max():.2f} of the tolerance"


def check_state(got, ref, E, what):
    err = (got.double().cpu() - ref).abs()
    tol = STEP * E[..., None] + 1e-30
    assert torch.isfinite(got).all(), what
    assert (err <= tol).all(), f"{what}: worst {(err / tol).max():.2f} of the tolerance"


def inputs(seed, T, Hk, Hv, D, strided=True, norm=True):
    """q, k, v (CPU, views of one tensor), g, beta; the same on the GPU."""
    gen = torch.Generator().manual_seed(seed)
    qkv = torch.randn(T, 2 * Hk + Hv, D, generator=gen)
    if not norm:                                    # keys no longer than 1, also after rounding
        qkv[:, :2 * Hk] /= 1.01 * qkv[:, :2 * Hk].norm(dim=-1, keepdim=True)
    qkv = qkv.to(torch.bfloat16)
    rate = torch.exp(torch.linspace(-7.0, 0.0, Hv))
    gb = torch.stack([-rate * torch.rand(T, Hv, generator=gen), torch.rand(T, Hv, generator=gen)], 1)
    d, e = qkv.cuda(), gb.cuda()
    parts = lambda x: (x[:, :Hk], x[:, Hk:2 * Hk], x[:, 2 * Hk:])  # noqa: E731
    dev = parts(d) + (e[:, 0], e[:, 1])
    if not strided:
        dev = tuple(x.contiguous() for x in dev)
    return parts(qkv) + (gb[:, 0], gb[:, 1]), dev, gen


def i32(*x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("lens,Hk,Hv,D,strided,norm", [
    ([1], 1, 1, 64, True, True), ([1], 2, 2, 128, False, False), ([63, 64, 65], 2, 2, 128, True, True),
    ([1, 2, 0, 3, 130], 2, 4, 64, True, False), ([200, 0, 1, 77], 1, 3, 128, True, True),
    ([129, 300], 2, 8, 64, False, True), ([512], 4, 4, 128, True, False), ([17] * 20, 4, 4, 64, True, True),
    ([1000, 5], 1, 2, 128, True, True), ([640], 2, 2, 64, True, False), ([5] * 9, 2, 4, 128, True, True),
    ([16, 15, 1], 1, 2, 64, False, True), ([191, 33, 128], 1, 1, 128, True, False)])
@pytest.mark.parametrize("cached", [False, True])
def test_packed_sequences_match_the_recurrence(lens, Hk, Hv, D, strided, norm, cached):
    B, T = len(lens), sum(lens)
    host, dev, gen = inputs(T + D, T, Hk, Hv, D, strided, norm)
    cu, scale, eps = cu_of(lens), D ** -0.5, 1e-6 if norm else None
    state = torch.randn(B + 2, Hv, D, D, generator=gen)
    slots = torch.randperm(B + 2, generator=gen)[:B].to(torch.int32)
    ctx = torch.tensor([b % 2 * 10 for b in range(B)], dtype=torch.int32)
    sd = state.cuda()
    av.get_last_device_error()
    kw = dict(state_cache=sd, state_slots=slots.cuda(), context_lens=ctx.cuda()) if cached else {}
    out = av.delta_attn_varlen_fwd(*dev, cu.cuda(), max(lens), scale, qk_norm_eps=eps, **kw)
    torch.cuda.synchronize()
    assert av.get_last_device_error()[0] == 0
    starts = [state[slots[b]].double() if cached and ctx[b] > 0 else None for b in range(B)]
    ref, finals, reach = delta(*host, cu, scale, starts, eps)
    check_out(out, ref, reach, "out")
    if cached:
        got = sd.cpu()
        for b in range(B):
            if lens[b] == 0:
                assert torch.equal(got[slots[b]], state[slots[b]])
            else:
                check_state(got[slots[b]], *finals[b], f"state {b}")
        free = [s for s in range(B + 2) if s not in slots.tolist()]
        assert torch.equal(got[free], state[free])


@pytest.mark.parametrize("B,Hk,Hv,D,strided,norm", [(1, 1, 1, 64, True, True), (3, 2, 8, 128, True, False),
                                                    (40, 4, 4, 64, False, True), (7, 1, 5, 128, True, True)])
def test_decode_matches_the_recurrence(B, Hk, Hv, D, strided, norm):
    host, dev, gen = inputs(B + D, B, Hk, Hv, D, strided, norm)
    scale, eps = 0.3, 1e-6 if norm else None
    state = torch.randn(B + 2, Hv, D, D, generator=gen)
    slots = torch.randperm(B + 2, generator=gen)[:B].to(torch.int32)
    if B > 2:
        slots[1] = -1
    ctx = torch.ones(B, dtype=torch.int32)
    ctx[::3] = 0
    for use_ctx in (False, True):
        sd = state.cuda()
        av.get_last_device_error()
        out = av.delta_attn_decode(*dev, sd, slots.cuda(), scale, context_lens=ctx.cuda() if use_ctx else None,
                                   qk_norm_eps=eps)
        torch.cuda.synchronize()
        assert av.get_last_device_error()[0] == 0
        starts = [state[slots[b]].double() if slots[b] >= 0 and not (use_ctx and ctx[b] == 0) else None
                  for b in range(B)]
        ref, finals, reach = delta(*host, list(range(B + 1)), scale, starts, eps)
        check_out(out, ref, reach, "out")
        got, want = sd.cpu(), state.clone()
        for b in range(B):
            if slots[b] >= 0:
                check_state(got[slots[b]], *finals[b], f"state {b}")
                want[slots[b]] = got[slots[b]]
        assert torch.equal(got, want)


@pytest.mark.parametrize("D", [64, 128])
def test_decays_and_strengths_at_the_ends_of_their_range(D):
    """No decay, a slow one over many chunks, one that is gone after a token, e^g = 0 in
    single tokens; beta 0 (nothing is written), 1 and in between."""
    lens, H = [450, 3], 4
    host, dev, _ = inputs(5, sum(lens), H, H, D)
    g, beta = host[3], host[4]
    for x, y in ((g, beta), dev[3:]):
        x[:, 0], x[:, 1], x[:, 2] = 0.0, -1e-4, -40.0
        x[::50, 3] = float("-inf")
        x[100:140, 3] = -300.0
        y[:, 0], y[:, 1] = 1.0, 0.5
        y[10:200:2, 2], y[60:250, 3] = 0.0, 0.0
    sd = torch.full((2, H, D, D), float("nan"), device="cuda")          # never read: both start from zero
    av.get_last_device_error()
    out = av.delta_attn_varlen_fwd(*dev, cu_of(lens).cuda(), 450, 1.0, state_cache=sd, state_slots=i32(1, 0),
                                   qk_norm_eps=0.0)
    torch.cuda.synchronize()
    assert av.get_last_device_error()[0] == 0
    ref, finals, reach = delta(*host, cu_of(lens), 1.0, [None, None], 0.0)
    check_out(out, ref, reach, "out")
    check_state(sd[1], *finals[0], "state")
    check_state(sd[0], *finals[1], "state")


def test_equal_keys_are_written_over():
    """The same key again and again: the inverse of the chunk's triangle is as far from a
    sum of few terms as it gets; with beta 1 the state holds the last value alone."""
    T, D = 200, 128
    host, dev, _ = inputs(8, T, 1, 2, D)
    for x in (host, dev):
        x[1][:] = x[1][0].clone()
        x[3][:] = 0.0
        x[4][:, 0], x[4][:, 1] = 1.0, 0.25
    s = torch.zeros(1, 2, D, D, device="cuda")
    out = av.delta_attn_varlen_fwd(*dev, i32(0, T), T, state_cache=s, state_slots=i32(0), qk_norm_eps=1e-6)
    ref, finals, reach = delta(*host, [0, T], D ** -0.5, [None], 1e-6)
    check_out(out, ref, reach, "out")
    check_state(s[0], *finals[0], "state")


def test_a_prompt_at_once_in_pieces_and_token_by_token_agree():
    T, D = 150, 128
    host, dev, _ = inputs(9, T, 1, 2, D)
    ref, finals, reach = delta(*host, [0, T], D ** -0.5, [None], 1e-6)
    for pieces in ([150], [1, 64, 20, 65], [149, 1], [70, 5, 5, 5, 65], [1] * 150):
        s = torch.full((1, 2, D, D), float("nan"), device="cuda")
        out, at = [], 0
        for n in pieces:
            x, past = [y[at:at + n] for y in dev], i32(at)
            if len(pieces) == T:
                out.append(av.delta_attn_decode(*x, s, i32(0), context_lens=past, qk_norm_eps=1e-6))
            else:
                out.append(av.delta_attn_varlen_fwd(*x, i32(0, n), n, state_cache=s, state_slots=i32(0),
                                                    context_lens=past, qk_norm_eps=1e-6))
            at += n
        check_out(torch.cat(out), ref, reach, str(len(pieces)))
        check_state(s[0], *finals[0], str(len(pieces)))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("lens", [[70, 33, 5], [6, 4, 5]])
def test_rows_of_other_sequences_and_behind_the_last_do_not_reach_a_sequence(D, lens):
    H, T = 2, sum(lens)
    a = cu_of(lens).tolist()
    host, dev, _ = inputs(3, T + 80, H, H, D, strided=False)
    for x in host + dev:
        x[a[1]:a[2]] = float("nan")
        x[a[1]:a[2]:2, ..., ::3] = float("inf")
        x[T:] = float("nan")
    out = torch.full((T + 80, H, D), 7.0, dtype=torch.bfloat16, device="cuda")
    sd = torch.full((5, H, D, D), float("nan"), device="cuda")
    av.delta_attn_varlen_fwd(*dev, cu_of(lens).cuda(), max(lens), 1.0, state_cache=sd, state_slots=i32(4, -1, 0),
                             out=out, qk_norm_eps=1e-6)
    torch.cuda.synchronize()
    for b, slot in ((0, 4), (2, 0)):
        ref, finals, reach = delta(*(x[a[b]:a[b + 1]] for x in host), [0, lens[b]], 1.0, [None], 1e-6)
        check_out(out[a[b]:a[b + 1]], ref, reach, f"sequence {b}")
        check_state(sd[slot], *finals[0], f"state {b}")
    assert out[T:].eq(7.0).all()
    assert sd[1:4].isnan().all()
    av.get_last_device_error()


@pytest.mark.parametrize("T", [9, 150])
@pytest.mark.parametrize("D", [64, 128])
def test_a_nan_reaches_later_tokens_alone(T, D):
    """One in v its value dimension from its token on, one in k or beta everything from its
    token on, one in q its own token's outputs; one infinity in v like a NaN."""
    at = T // 2
    for which in ("v", "inf", "k", "q", "beta"):
        host, dev, _ = inputs(11, T, 2, 2, D)
        clean = [x.clone() for x in host]
        i = {"q": 0, "k": 1, "v": 2, "inf": 2, "beta": 4}[which]
        bad = float("inf") if which == "inf" else float("nan")
        if which == "beta":
            dev[i][at, 1] = bad
        else:
            dev[i][at, 1, 5] = bad
        s = torch.zeros(1, 2, D, D, device="cuda")
        out = av.delta_attn_varlen_fwd(*dev, i32(0, T), T, state_cache=s, state_slots=i32(0), qk_norm_eps=1e-6)
        ref, finals, (rm, re) = delta(*clean, [0, T], D ** -0.5, [None], 1e-6)
        hit = torch.zeros(T, 2, D, dtype=torch.bool)
        if which == "q":
            hit[at, 1] = True
        elif i == 2:
            hit[at:, 1, 5] = True
        else:
            hit[at:, 1] = True
        got = out.cpu()
        assert not torch.isfinite(got[hit].float()).any(), which
        check_out(got[~hit], ref[~hit], (rm[~hit], re[~hit]), which)
        got, bad_rows = s[0].cpu(), hit[-1] if which != "q" else torch.zeros(2, D, dtype=torch.bool)
        assert not torch.isfinite(got[bad_rows]).any(), which
        S, E = finals[0]
        check_state(got[~bad_rows], S[~bad_rows], E[~bad_rows], which)
        av.get_last_device_error()


def test_bad_indices_decays_and_refused_entries():
    D, H = 64, 2
    run = functools.partial(av.delta_attn_varlen_fwd, qk_norm_eps=1e-6)     # (longer keys diverge)
    for n in (8, 100):                                       # the short form and the chunked one
        host, dev, _ = inputs(4, 2 * n, H, H, D)
        sd = torch.zeros(2, H, D, D, device="cuda")
        av.get_last_device_error()
        # offsets past the tokens, decreasing offsets
        out = torch.full((2 * n, H, D), 7.0, dtype=torch.bfloat16, device="cuda")
        run(*dev, i32(0, n, n // 2, 4 * n), n, state_cache=sd, state_slots=i32(0, 1, 1), out=out)
        assert av.get_last_device_error()[0] == 6
        assert out[n:].eq(7.0).all() and not out[:n].eq(7.0).all() and sd[1].eq(0).all()
        # a slot past the cache: the sequence runs from zero and keeps nothing
        a = run(*dev, i32(0, 2 * n), 2 * n, state_cache=sd, state_slots=i32(2),
                                     context_lens=i32(5))
        assert av.get_last_device_error()[0] == 6
        b = run(*dev, i32(0, 2 * n), 2 * n)
        assert torch.equal(a, b) and sd[1].eq(0).all()
        # longer than max_seqlen: cut to it
        out.fill_(7.0)
        run(*dev, i32(0, 2 * n), n, out=out)
        assert av.get_last_device_error()[0] == 6
        assert torch.equal(out[:n], b[:n]) and out[n:].eq(7.0).all()
        # a positive decay and a NaN one count as none
        g = dev[3].clone()
        g[3, 0], g[5, 1] = 2.0, float("nan")
        got = run(*dev[:3], g, dev[4], i32(0, 2 * n), 2 * n)
        assert av.get_last_device_error()[0] == 8
        g[3, 0], g[5, 1] = 0.0, 0.0
        assert torch.equal(got, run(*dev[:3], g, dev[4], i32(0, 2 * n), 2 * n))
        # refused entries run from zero and leave their states
        sd = torch.randn(2, H, D, D, device="cuda")
        kept = sd.clone()
        got = run(*dev, i32(0, n, 2 * n), n, state_cache=sd, state_slots=i32(0, 1),
                                       context_lens=i32(7, 7), cache_seqlens=i32(7, 7 + n))
        assert av.get_last_device_error()[0] == 0
        assert torch.equal(got[:n], run(*(x[:n] for x in dev), i32(0, n), n))
        assert torch.equal(sd[0], kept[0]) and not torch.equal(sd[1], kept[1])


@pytest.mark.parametrize("T", [5, 300])
def test_captured_replayed_and_repeated(T):
    """Bit-equal each time, as one graph and on a stream of its own."""
    D, Hk, Hv = 128, 2, 4
    host, dev, gen = inputs(13, T, Hk, Hv, D)
    start = torch.randn(3, Hv, D, D, generator=gen).cuda()
    kw = dict(state_slots=i32(2), context_lens=i32(9), qk_norm_eps=1e-6)
    s0 = start.clone()
    want = av.delta_attn_varlen_fwd(*dev, i32(0, T), T, state_cache=s0, **kw)
    cu, state, out = i32(0, T), start.clone(), torch.empty_like(want)
    ws = torch.empty(max(1, av.delta_attn_workspace_size(1, T, Hk, Hv, D, T)), dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            av.delta_attn_varlen_fwd(*dev, cu, T, state_cache=state, out=out, workspace=ws, **kw)
        for _ in range(3):
            out.zero_()
            state.copy_(start)
            graph.replay()
            side.synchronize()
            assert torch.equal(out, want) and torch.equal(state, s0)
    state.copy_(start)
    torch.cuda.synchronize()
    again = av.delta_attn_varlen_fwd(*dev, cu, T, state_cache=state, stream=side, **kw)
    side.synchronize()
    assert torch.equal(again, want) and torch.equal(state, s0)
    assert av.get_last_device_error()[0] == 0


@pytest.mark.parametrize("lens,Hk,Hv,D", [([3000], 1, 1, 128), ([2100, 70, 1700, 0, 3], 1, 2, 64), ([640, 1800], 1, 1, 64),
                                          ([20, 2561], 2, 2, 128)])
@pytest.mark.parametrize("cached", [False, True])
def test_long_sequences_cut_into_segments(lens, Hk, Hv, D, cached):
    """Fewer sequences and heads than the GPU has room for: segments run side by side from the
    states that a pass before finds (a matrix per segment, applied to its start: sums of D terms, whose
    rounding of D 2^-24 at most per segment the steps' allowance covers: a segment has 512 tokens at least)."""
    B, T = len(lens), sum(lens)
    assert av.delta_attn_workspace_size(B, T, Hk, Hv, D, max(lens)) > 1 << 20          # it does cut them
    host, dev, gen = inputs(T, T, Hk, Hv, D)
    cu = cu_of(lens)
    state = torch.randn(B + 1, Hv, D, D, generator=gen)
    slots = torch.randperm(B + 1, generator=gen)[:B].to(torch.int32)
    ctx = torch.tensor([7] * B, dtype=torch.int32)
    sd = state.cuda()
    av.get_last_device_error()
    kw = dict(state_cache=sd, state_slots=slots.cuda(), context_lens=ctx.cuda()) if cached else {}
    out = av.delta_attn_varlen_fwd(*dev, cu.cuda(), max(lens), qk_norm_eps=1e-6, **kw)
    torch.cuda.synchronize()
    assert av.get_last_device_error()[0] == 0
    ref, finals, reach = delta(*host, cu, D ** -0.5, [state[slots[b]].double() if cached else None for b in range(B)], 1e-6)
    check_out(out, ref, reach, "out")
    if cached:
        for b in range(B):
            if lens[b]:
                check_state(sd[slots[b]], *finals[b], f"state {b}")
        free = [s for s in range(B + 1) if s not in slots.tolist()] + [int(slots[b]) for b in range(B) if lens[b] == 0]
        assert torch.equal(sd.cpu()[free], state[free])


@pytest.mark.parametrize("lens", [[2, 1, 0, 2], [7, 8, 3], [9, 1, 8], [12, 16, 0, 5, 15], [32, 17, 31, 1], [33, 96, 40]])
@pytest.mark.parametrize("Hk,Hv,D", [(2, 2, 64), (1, 3, 128), (2, 4, 128)])
@pytest.mark.parametrize("strided", [False, True])
def test_lengths_around_the_forms_limits(lens, Hk, Hv, D, strided):
    """Up to 8 and up to 16 tokens in one pass over the states, up to 32 and more in chunks; decays and strengths at
    the ends of their range among them.  One pass: products of the state and of u as parts of 2^-24 together, summed in fp32
    over D terms and up to 16 tokens (the step's 128 x 2^-24 covers both); outputs take the state as two parts, 2^-16
    of scale |q| M."""
    B, T = len(lens), sum(lens)
    host, dev, gen = inputs(7 * T + D, T, Hk, Hv, D, strided, True)
    g, beta = host[3].clone(), host[4].clone()
    g[::5, 0], g[3::7, -1], beta[1::4, 0], beta[2::4, -1] = float("-inf"), 0.0, 0.0, 1.0
    host, dev = (*host[:3], g, beta), (*dev[:3], g.cuda(), beta.cuda())
    cu, scale = cu_of(lens), D ** -0.5
    state = torch.randn(B + 1, Hv, D, D, generator=gen)
    slots = torch.randperm(B + 1, generator=gen)[:B].to(torch.int32)
    ctx = torch.tensor([0 if b == 1 else 5 for b in range(B)], dtype=torch.int32)
    sd = state.cuda()
    av.get_last_device_error()
    out = av.delta_attn_varlen_fwd(*dev, cu.cuda(), max(lens), scale, state_cache=sd, state_slots=slots.cuda(),
                                   context_lens=ctx.cuda(), qk_norm_eps=1e-6)
    torch.cuda.synchronize()
    assert av.get_last_device_error()[0] == 0
    starts = [state[slots[b]].double() if ctx[b] > 0 else None for b in range(B)]
    ref, finals, reach = delta(*host, cu, scale, starts, 1e-6)
    check_out(out, ref, reach, "out")
    got = sd.cpu()
    for b in range(B):
        if lens[b] == 0:
            assert torch.equal(got[slots[b]], state[slots[b]])
        else:
            check_state(got[slots[b]], *finals[b], f"state {b}")
    free = [s for s in range(B + 1) if s not in slots.tolist()]
    assert torch.equal(got[free], state[free])
    # the same bits each time
    again = state.cuda()
    assert torch.equal(out, av.delta_attn_varlen_fwd(*dev, cu.cuda(), max(lens), scale, state_cache=again,
                                                     state_slots=slots.cuda(), context_lens=ctx.cuda(), qk_norm_eps=1e-6))
    assert torch.equal(again, sd)


@pytest.mark.parametrize("T", [2, 6, 16, 20, 40])
@pytest.mark.parametrize("D", [64, 128])
def test_a_nan_in_every_form(T, D):
    test_a_nan_reaches_later_tokens_alone(T, D)
