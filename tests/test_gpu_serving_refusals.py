"""A step in which a request is refused (its row has no room for its pages): what
the layers compute and keep for the others."""
import numpy as np
import pytest
import torch

import attention_attn_varlen_gb300 as av
import oracle
from attention_attn_varlen_gb300.attention import Attention, LinearAttention, PagePool
from _util import assert_close

pytestmark = pytest.mark.gpu

Hq, Hkv, D, BS, M = 8, 2, 64, 16, 4          # a row holds 64 tokens


def _i32(*x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _attend(q, k, v):
    """Causal attention of the last len(q) of len(k) tokens, in 64 bits."""
    i32 = lambda *x: np.asarray(x, dtype=np.int32)  # noqa: E731
    out, _ = oracle.attn_varlen(q, k, v, i32(0, len(q)), i32(0, len(k)), Hq, Hkv, D, D ** -0.5, True)
    return out.reshape(q.shape)


@pytest.mark.parametrize("where", [0, 1])
def test_a_refused_prompt_leaves_the_other_one_its_own_keys(where):
    gen = torch.Generator().manual_seed(3)
    mk = lambda n: [torch.randn(n, h, D, generator=gen).to(torch.bfloat16) for h in (Hq, Hkv, Hkv)]  # noqa: E731
    pool = PagePool(40, BS, 3, M)
    att = Attention(Hq, D, D ** -0.5, Hkv)
    att.k_cache, att.v_cache = (torch.zeros(40, BS, Hkv, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    av.get_last_device_error()
    hist = None
    for kind, served in (("fresh", 20), ("paged", 7)):
        new = [served, served]
        new[where] = 100                      # more than a row's pages hold
        rows = [2, 2]
        rows[where] = 0
        x = mk(sum(new))
        t = pool.grow(_i32(*new), sum(new), request_rows=_i32(*rows))
        ctx = pool.context(t, True, max(new), 128, paged=kind == "paged")
        o = att(*(y.cuda() for y in x), ctx).cpu()
        assert av.get_last_device_error()[0] == 9
        mine = slice(0, served) if where == 1 else slice(100, 100 + served)
        own = [y[mine] for y in x]
        hist = own[1:] if hist is None else [torch.cat(y) for y in zip(hist, own[1:])]
        assert_close(o[mine], _attend(own[0], *hist), kind)
        pages = t.block_table[1 - where].long()
        n = len(hist[0])
        for cache, want in zip((att.k_cache, att.v_cache), hist):
            assert torch.equal(cache[pages[:-(-n // BS)]].view(-1, Hkv, D)[:n].cpu(), want), kind
    assert pool.seq_lens.tolist() == [0, 0, 27]


@pytest.mark.parametrize("Hq,Hkv,D", [(2, 2, 64), (4, 1, 128)])
@pytest.mark.parametrize("new,refused", [([1, 1, 1, 1], [1, 3]), ([5, 70, 1, 0], [1]), ([2000, 9, 40, 3000], [0]),
                                         ([2000, 9, 40, 3000], [3]), ([3, 3, 3, 3], [0, 1, 2, 3])])
def test_a_refused_request_keeps_its_linear_state(Hq, Hkv, D, new, refused):
    """Its tokens run all the same, and nothing of them is kept.  The others have the bits of a
    step that serves everyone."""
    B, T = len(new), sum(new)
    gen = torch.Generator(device="cuda").manual_seed(T)
    rnd = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    q, k, v = (rnd(T, h, D).bfloat16() for h in (Hq, Hkv, Hkv))
    state = rnd(B, Hkv, D, D)
    g = torch.linspace(-0.5, -0.001, Hkv, device="cuda")
    slots, rows = _i32(2, 0, 3, 1), _i32(*range(B))
    past = [3, 0, 40, 7]

    def run(full):
        pool = PagePool(1000, BS, B, 400)
        pool.grow(_i32(*past), sum(past))
        for b in full:                                    # rows as long as they may get
            pool.seq_lens[b] = 400 * BS
            pool.page_table[b] = 0
        t = pool.grow(_i32(*new), T)
        lin = LinearAttention(Hq, D, D ** -0.5, Hkv, g)
        lin.state_cache = state.clone()
        y = lin(q, k, v, pool.context(t, max(new) > 1, max(new), 400 * BS, state_slots=slots))
        return t, y, lin.state_cache

    av.get_last_device_error()
    t, y, got = run(refused)
    assert av.get_last_device_error()[0] == 9
    _, want_y, want = run([])
    assert av.get_last_device_error()[0] == 0
    cu = t.cu_seqlens_q.tolist()
    for b in range(B):
        s = slots[b].item()
        if b in refused or new[b] == 0:
            assert torch.equal(got[s], state[s]), b
        else:
            assert torch.equal(got[s], want[s]) and torch.equal(y[cu[b]:cu[b + 1]], want_y[cu[b]:cu[b + 1]]), b
            assert not torch.equal(got[s], state[s])
