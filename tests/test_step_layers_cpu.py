"""What the layers make of a step's tables, on a machine without a GPU: which
call they route to, with which offsets and rows."""
import pytest
import torch

import attention_attn_varlen_gb300 as av
import attention_attn_varlen_gb300.attention as at


def _i32(*x):
    return torch.tensor(x, dtype=torch.int32)


def _tables(context, new, served):
    """The tables of a step as step_tables writes them, without pages."""
    after = [c + n if s else c for c, n, s in zip(context, new, served)]
    cu = lambda x: _i32(0, *torch.tensor(x).cumsum(0).tolist())  # noqa: E731
    return av.StepTables(_i32(*[-1] * len(new)).view(-1, 1), torch.arange(sum(new)), _i32(*range(sum(new))), cu(new),
                         cu(after), _i32(*after), _i32(*context))


def test_fresh_prompts_read_their_own_rows_whoever_was_served():
    """100 and 20 tokens, the first prompt refused: its rows still stand in q, k and v."""
    t = _tables([0, 0], [100, 20], [False, True])
    assert t.cu_seqlens_k.tolist() == [0, 0, 20]
    ctx = at.PagePool.context(t, True, 100, 128, paged=False)
    assert ctx.cu_seqlens_q.tolist() == ctx.cu_seqlens_k.tolist() == [0, 100, 120]
    assert ctx.max_seqlen_k == 100 and ctx.block_tables is None
    ctx = at.PagePool.context(t, True, 100, 128)
    assert ctx.cu_seqlens_k is t.cu_seqlens_k and ctx.max_seqlen_k == 128 and ctx.block_tables is t.block_table


@pytest.fixture
def linear(monkeypatch):
    """A layer with states of four slots, and the calls it makes."""
    calls = []

    def note(name):
        def f(q, k, v, g, *a, **kw):
            calls.append((name, a, kw))
            return torch.zeros_like(q)
        return f

    for name in ("linear_attn_decode", "linear_attn_varlen_fwd"):
        monkeypatch.setattr(at, name, note(name))
    layer = at.LinearAttention(2, 64, 0.5, 1, torch.zeros(1))
    layer.state_cache = torch.zeros(4, 1, 64, 64)

    def run(ctx, rows):
        calls.clear()
        layer(torch.zeros(rows, 128), torch.zeros(rows, 64), torch.zeros(rows, 64), ctx)
        return calls[0]
    return run


@pytest.mark.parametrize("new,pad", [([2, 0], 0), ([3, 1, 0, 0], 0), ([1, 0, 1, 1], 1), ([1, 0, 1], 0), ([2, 0, 1], 0),
                                     ([1, 1, 1], 0), ([1, 1, 0], 2), ([2, 2], 0)])
def test_a_decode_step_goes_by_its_offsets(linear, new, pad):
    """As many rows as sequences is no sign of one token each: rows are packed in entry
    order, so that an entry without a token moves the ones behind it."""
    B = len(new)
    t = _tables([5] * B, new, [True] * B)
    ctx = at.PagePool.context(t, False, max(new), 64, state_slots=torch.arange(B).int())
    name, a, kw = linear(ctx, sum(new) + pad)
    assert name == "linear_attn_varlen_fwd" and a[0] is t.cu_seqlens_q and a[1] == max(new)
    assert kw["state_slots"] is ctx.state_slots and kw["context_lens"] is t.context_lens


def test_the_linear_layer_hears_who_was_served(linear):
    t = _tables([5, 0, 7], [1, 1, 1], [True, False, True])
    for prefill in (False, True):
        ctx = at.PagePool.context(t, prefill, 1, 64, state_slots=_i32(0, 1, 2))
        assert ctx.cache_seqlens is t.cache_seqlens
        name, a, kw = linear(ctx, 3)
        assert name == "linear_attn_varlen_fwd" and kw["cache_seqlens"] is t.cache_seqlens
    ctx = at.AttentionContext(True, state_slots=_i32(0, 1, 2), cu_seqlens_q=_i32(0, 1, 1, 2), max_seqlen_q=1,
                              context_lens=_i32(1, 1, 1))
    assert linear(ctx, 3)[2]["cache_seqlens"] is None    # contexts made by hand say nothing about it


def test_a_decode_step_without_offsets_has_a_row_for_each_sequence(linear):
    slots, past = _i32(2, 0, 1), _i32(4, 4, 4)
    ctx = at.AttentionContext(False, state_slots=slots, past_lens=past)
    name, a, kw = linear(ctx, 3)
    assert name == "linear_attn_decode" and a[1] is slots and kw["context_lens"] is past
    with pytest.raises(ValueError, match="offsets"):
        linear(ctx, 4)
    # offsets, and no word on what came before: every slot continues, as without offsets
    ctx = at.AttentionContext(False, state_slots=slots, cu_seqlens_q=_i32(0, 1, 1, 2), max_seqlen_q=1)
    name, a, kw = linear(ctx, 3)
    assert name == "linear_attn_varlen_fwd" and kw["context_lens"].tolist() == [1, 1, 1]
    # no bound on the counts either
    ctx = at.AttentionContext(False, state_slots=slots, cu_seqlens_q=_i32(0, 2, 2, 3), past_lens=past)
    name, a, kw = linear(ctx, 3)
    assert name == "linear_attn_varlen_fwd" and a[1] == 3


def test_sequences_of_at_most_one_token_need_no_workspace():
    av.build()
    L = av.lib()
    assert L.attn_linear_workspace_size(256, 32, 8, 128, 1) == L.attn_linear_workspace_size(256, 32, 8, 128, 0) == 0
    assert L.attn_linear_workspace_size(256, 32, 8, 128, 2) > 0
    if torch.cuda.is_available():
        return                                           # made-up addresses below: they must find no device
    call = lambda most: L.attn_linear_varlen_fwd(0x1000, 0x1000, 0x1000, 0x1000, 0x1000, 0x1000, None, None, None, 4,  # noqa: E731
                                                 4, most, 2, 1, 64, 0.1, 0, 0, 0, 0, 0, None, 0, None)
    assert call(1) == 7 and call(2) == 1 and call(0) == 0


@pytest.mark.skipif(torch.cuda.is_available(), reason="passes made-up device addresses")
def test_the_entry_for_a_steps_entries_checks_what_the_plain_one_does():
    av.build()
    L = av.lib()
    F = 0x1000

    def call(B=2, Hq=4, Hkv=2, D=64, state=F, slots=F, after=F, most=8, ws_bytes=1 << 40, qs=0, cu=F):
        return L.attn_linear_step_fwd(F, F, F, F, F, cu, state, slots, None, after, B, 10, most, Hq, Hkv, D, 0.1, 4, qs,
                                      0, 0, 0, F, ws_bytes, None)

    assert call() == call(after=None) == call(state=None, slots=None) == 7
    assert call(cu=None) == call(Hq=3) == call(state=None) == call(qs=4) == call(most=-1) == 1
    assert call(D=96) == 2 and call(ws_bytes=8) == 3 and call(ws_bytes=0, most=1) == 7 and call(most=0) == 0
