"""A step in which a request is refused (its row has no room for its pages): what
the layers compute and keep for the others."""
import numpy as np
import pytest
import torch

import attention_attn_varlen_gb300 as av
import oracle
from attention_attn_varlen_gb300.attention import Attention, PagePool
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
