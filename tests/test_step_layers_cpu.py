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
