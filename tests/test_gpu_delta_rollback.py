"""Guessed tokens that are accepted in part, through DeltaAttention: the states are saved in spare
slots, the step runs over all tokens, and where not all are accepted the saved states come back and
the layer runs again over the accepted ones.  Outputs and states against the recurrence over the
accepted history, in 64 bits, with the tolerances of the rule's other tests."""
import pytest
import torch

import attention_attn_varlen_gb300 as av
from attention_attn_varlen_gb300.attention import AttentionContext, DeltaAttention
from _delta_reference import delta
from _step_reference import cu_of
from test_gpu_delta_attn import check_out, check_state, i32


def test_cut_workspaces_are_not_empty():
    """Sizes for which a workspace's refusals are tested elsewhere do need one."""
    av.build()
    assert av.delta_attn_workspace_size(2, 10, 2, 4, 64, 100) > 0
    assert av.delta_attn_workspace_size(2, 10, 2, 4, 64, 16) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("guessed,accepted", [(5, [3, 1, 5, 2]), (5, [1, 1, 1, 1]), (5, [5, 5, 5, 5]), (16, [7, 16, 1, 9]),
                                              (3, [0, 3, 0, 1]), (40, [17, 40, 0, 33])])
@pytest.mark.parametrize("D", [64, 128])
def test_guessed_tokens_accepted_in_part(guessed, accepted, D):
    Hk, Hv, B = 1, 2, 4
    gen = torch.Generator().manual_seed(guessed + D)
    layer = DeltaAttention(Hk, Hv, D, D ** -0.5)
    layer.state_cache = torch.full((2 * B, Hv, D, D), float("nan"), device="cuda")
    rows, spare = i32(2, 0, 3, 1), i32(4, 5, 6, 7)

    def tokens(n):
        qkv = torch.randn(n, 2 * Hk + Hv, D, generator=gen).to(torch.bfloat16)
        return [qkv[:, :Hk], qkv[:, Hk:2 * Hk], qkv[:, 2 * Hk:], -0.2 * torch.rand(n, Hv, generator=gen),
                torch.rand(n, Hv, generator=gen)]

    def step(x, new, past, prefill=False):
        dev = [y.contiguous().cuda() for y in x]
        return layer(*dev, AttentionContext(prefill, cu_seqlens_q=cu_of(new).cuda(), max_seqlen_q=max(new), state_slots=rows,
                                            past_lens=i32(*past)))

    def check(out, x, new, starts, what):
        ref, finals, reach = delta(*x, cu_of(new), D ** -0.5, starts, 1e-6)
        check_out(out, ref, reach, what)
        return finals

    av.get_last_device_error()
    lens = [70, 1, 129, 20]
    x = tokens(sum(lens))
    finals = check(step(x, lens, [0] * B, True), x, lens, [None] * B, "prompts")
    states = [layer.state_cache[int(r)].double().cpu() for r in rows]
    for b in range(B):
        check_state(states[b], *finals[b], "prompt")
    past = lens
    for turn in range(3):
        x = tokens(guessed * B)
        av.copy_states(layer.state_cache, rows, spare)
        check(step(x, [guessed] * B, past), x, [guessed] * B, states, "guessed")
        # the sequences that keep all of their tokens need nothing; -1: not copied
        part = torch.tensor([a < guessed for a in accepted], device="cuda")
        av.copy_states(layer.state_cache, torch.where(part, spare, -1), rows)
        again = [a if a < guessed else 0 for a in accepted]
        own = [torch.cat([y[b * guessed:b * guessed + again[b]] for b in range(B)]) for y in x]
        if sum(again):
            check(step(own, again, past), own, again, states, "again")
        kept = [torch.cat([y[b * guessed:b * guessed + accepted[b]] for b in range(B)]) for y in x]
        finals = delta(*kept, cu_of(accepted), D ** -0.5, states, 1e-6)[1]
        for b in range(B):
            got = layer.state_cache[int(rows[b])]
            if accepted[b]:
                check_state(got, *finals[b], f"turn {turn}")
            else:
                assert torch.equal(got.double().cpu(), states[b])
            states[b] = got.double().cpu()
        past = [p + a for p, a in zip(past, accepted)]
        accepted = accepted[1:] + accepted[:1]
    assert av.get_last_device_error()[0] == 0
