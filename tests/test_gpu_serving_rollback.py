"""Speculative tokens that are accepted in part: both layers run over all of them, then
the pages behind the accepted ones go back, the linear layer's states are put back and
run again over the accepted tokens; padding rows on the way.  Against 64-bit references
over the accepted history, and a plain pool, integer by integer.

Tolerances as in the other step tests: attention against the float64 oracle; linear
attention 2^-8 of the output and 2^-13 of the terms' absolute values for outputs and
states (two bf16 parts of a term, and what a few hundred steps add up to)."""
import numpy as np
import pytest
import torch

import attention_attn_varlen_gb300 as av
import oracle
from attention_attn_varlen_gb300.attention import Attention, AttentionContext, LinearAttention, PagePool, Rotary
from _step_reference import Pool, cu_of, linear, rope
from _util import assert_close

pytestmark = pytest.mark.gpu

Hq, Hkv, D, BS, R, M, PAGES = 8, 2, 64, 16, 4, 20, 50


class _Model:
    """An attention and a linear layer over one pool, and their whole history."""

    def __init__(self):
        self.gen = torch.Generator().manual_seed(21)
        self.pool, self.ref = PagePool(PAGES, BS, R, M), Pool([0] * R, [[-1] * M] * R, range(PAGES - 1, -1, -1), PAGES, BS)
        self.inv = (10000.0 ** (-torch.arange(D // 2, dtype=torch.float64) / (D // 2))).float()
        self.g = torch.tensor([-0.3, -0.01])
        self.att = Attention(Hq, D, D ** -0.5, Hkv, rotary=Rotary(self.inv.cuda()))
        self.att.k_cache = torch.full((PAGES, BS, Hkv, D), float("nan"), dtype=torch.bfloat16, device="cuda")
        self.att.v_cache = torch.full_like(self.att.k_cache, float("nan"))
        self.lin = LinearAttention(Hq, D, D ** -0.5, Hkv, self.g.cuda())
        self.lin.state_cache = torch.full((R, Hkv, D, D), float("nan"), device="cuda")
        none = torch.empty(0, Hkv, D, dtype=torch.bfloat16)
        self.hist = {r: [none, none] for r in range(R)}               # rotated k, v of each request's cached tokens
        self.states = {r: None for r in range(R)}                     # its state, in 64 bits

    def tokens(self, n):
        return [torch.randn(n, h, D, generator=self.gen).to(torch.bfloat16) for h in (Hq, Hkv, Hkv)]

    def grow(self, rows, new, T):
        t = self.pool.grow(_i32(new), T, request_rows=_i32(rows))
        want = self.ref.grow(rows, new, T)
        for f in av.StepTables._fields:
            assert getattr(t, f).tolist() == want[f], f
        self.same_pool()
        return t

    def trim(self, rows, keep):
        self.pool.trim(_i32(keep), request_rows=_i32(rows))
        self.ref.trim(rows, keep)
        self.same_pool()

    def same_pool(self):
        p, r = self.pool, self.ref
        assert p.seq_lens.tolist() == r.lens and p.page_table.tolist() == r.table
        assert p.num_free.item() == r.nf and p.free_pages.tolist()[:r.nf] == r.free[:r.nf]

    def attended(self, o, x, rows, new, what):
        """Check the attention of a step's tokens and add them to the history."""
        cu = cu_of(new).tolist()
        for b, r in enumerate(rows):
            if new[b] == 0:
                continue
            own = slice(cu[b], cu[b + 1])
            p = torch.arange(len(self.hist[r][0]), len(self.hist[r][0]) + new[b])[None]
            q, k = (rope(y[own], p, self.inv, None, False, 1.0).to(torch.bfloat16) for y in x[:2])
            self.hist[r] = [torch.cat(y) for y in zip(self.hist[r], (k, x[2][own]))]
            i32 = lambda *y: np.asarray(y, dtype=np.int32)  # noqa: E731
            want, _ = oracle.attn_varlen(q, *self.hist[r], i32(0, new[b]), i32(0, len(self.hist[r][0])), Hq, Hkv, D,
                                         D ** -0.5, True)
            assert_close(o[own], want.reshape(q.shape), what)

    def advanced(self, y, x, rows, new, what, keep=True):
        """Check the linear layer's outputs and states; keep: they are the history's from here on."""
        n = sum(new)
        want, finals, weight = linear(*(z[:n] for z in x), self.g, cu_of(new), D ** -0.5, [self.states[r] for r in rows])
        assert ((y[:n].double().cpu() - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -13 * weight).all(), what
        for (S, A), r, m in zip(finals, rows, new):
            if m:
                assert ((self.lin.state_cache[r].double().cpu() - S).abs() <= 2.0 ** -13 * A).all(), what
                if keep:
                    self.states[r] = self.lin.state_cache[r].double().cpu()

    def step(self, rows, new, kind, pad=0):
        n = sum(new)
        x = self.tokens(n + pad)
        for y in x:
            y[n:] = float("nan")                                      # padding rows hold anything
        t = self.grow(rows, new, n + pad)
        ctx = self.pool.context(t, kind != "decode", max(new), BS * M, paged=kind != "prompt", state_slots=_i32(rows))
        dev = [y.cuda() for y in x]
        self.attended(self.att(*dev, ctx).cpu(), x, rows, new, kind)
        self.advanced(self.lin(*dev, ctx), x, rows, new, kind)


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("accepted", [[3, 1], [0, 4], [4, 4], [0, 0]])
def test_speculative_tokens_accepted_in_part(accepted):
    m = _Model()
    av.get_last_device_error()
    m.step([0, 2, 3], [37, 126, 5], "prompt")
    m.step([2, 3, 0], [17, 0, 26], "prefix", pad=5)
    rows, past = [2, 0], [143, 63]
    # four guessed tokens each: the pages, and both layers over all of them
    kept, free = m.lin.state_cache.clone(), m.ref.nf
    x, t = m.tokens(8), m.grow(rows, [4, 4], 8)
    assert m.ref.nf == free - 2                                       # 143 + 4 and 63 + 4 tokens: a page each
    ctx = m.pool.context(t, False, 4, BS * M, state_slots=_i32(rows))
    dev = [y.cuda() for y in x]
    before = {r: m.hist[r] for r in rows}
    m.attended(m.att(*dev, ctx).cpu(), x, rows, [4, 4], "guessed")
    m.advanced(m.lin(*dev, ctx), x, rows, [4, 4], "guessed", keep=False)
    for r in range(R):
        assert torch.equal(m.lin.state_cache[r].nan_to_num(), kept[r].nan_to_num()) == (r not in rows), r
    # back to the accepted ones: the pages, the history, the states
    m.trim(rows, [p + a for p, a in zip(past, accepted)])
    assert m.ref.nf == free - sum(-(-(p + a) // BS) + -p // BS for p, a in zip(past, accepted))
    for r, a in zip(rows, accepted):
        m.hist[r] = [y[:len(z) + a] for y, z in zip(m.hist[r], before[r])]
    m.lin.state_cache.copy_(kept)
    if sum(accepted):
        pick = [4 * b + i for b in range(2) for i in range(accepted[b])]
        own = [y[pick] for y in x]
        redo = AttentionContext(False, cu_seqlens_q=cu_of(accepted).cuda(), max_seqlen_q=max(accepted),
                                state_slots=_i32(rows), past_lens=_i32(past))
        m.advanced(m.lin(*(y.cuda() for y in own), redo), own, rows, accepted, "accepted")
    m.step([0, 2, 3], [1, 1, 1], "decode")
    m.step([3, 0, 2], [40, 1, 17], "prefix", pad=3)
    m.trim([2], [0])
    m.hist[2], m.states[2] = [y[:0] for y in m.hist[2]], None
    m.step([2, 1], [33, 64], "prompt")
    m.step([0, 1, 2, 3], [1, 1, 1, 1], "decode")
    assert av.get_last_device_error()[0] == 0
