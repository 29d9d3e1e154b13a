"""A beam search as it runs in a model with attention and delta-rule layers: prompts,
steps, selection, rows that change hands, states and cached rows that follow them;
against every beam's own history, in 64 bits.

The choice is exact (on the step's own logits).  Cached keys and values are the tokens' own
bits.  States: the steps' allowance of the delta-rule tests, 128 x 2^-24 of what a row can
reach; outputs: attention against the float64 oracle, the delta rule as in its own tests."""
import numpy as np
import pytest
import torch

import attention_attn_varlen_gb300 as av
import oracle
from attention_attn_varlen_gb300.attention import Attention, Beams, DeltaAttention, LinearAttention, PagePool
from _delta_reference import delta, select
from _step_reference import cu_of, linear
from _util import assert_close

pytestmark = pytest.mark.gpu

HQ, HKV, HK, HV, D, BS, M, VOCAB = 4, 2, 1, 2, 64, 16, 8, 97


class _Model:
    """Fixed projections of every token; its layers' outputs give the logits."""

    def __init__(self, rows):
        gen = torch.Generator().manual_seed(77)
        randn = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
        self.qkv = randn(VOCAB, HQ + 2 * HKV, D).to(torch.bfloat16)
        self.dqkv = randn(VOCAB, 2 * HK + HV, D).to(torch.bfloat16)
        self.g, self.beta = -0.3 * torch.rand(VOCAB, HV, generator=gen), torch.rand(VOCAB, HV, generator=gen)
        self.head = randn((HQ + HV + HKV) * D, VOCAB).cuda()
        self.pool = PagePool(rows * M, BS, rows, M)
        self.att = Attention(HQ, D, D ** -0.5, HKV)
        self.att.k_cache = torch.full((rows * M, BS, HKV, D), float("nan"), dtype=torch.bfloat16, device="cuda")
        self.att.v_cache = torch.full_like(self.att.k_cache, float("nan"))
        self.att.v16_cache = torch.full(self.att.k_cache.shape, float("nan"), dtype=torch.float16, device="cuda")
        self.rule = DeltaAttention(HK, HV, D, D ** -0.5)
        self.rule.state_cache = torch.full((rows, HV, D, D), float("nan"), device="cuda")
        self.decay = torch.tensor([-0.2, -0.02])
        self.lin = LinearAttention(HKV, D, D ** -0.5, HKV, self.decay.cuda())
        self.lin.state_cache = torch.full((rows, HKV, D, D), float("nan"), device="cuda")
        self.layers = (self.att, self.rule, self.lin)
        self.dev = [x.cuda() for x in (self.qkv, self.dqkv, self.g, self.beta)]

    def run(self, tokens, ctx):
        """Outputs of the layers (packed) and the logits of every token."""
        qkv, dqkv, g, beta = (x[tokens.long()] for x in self.dev)
        a = self.att(qkv[:, :HQ], qkv[:, HQ:HQ + HKV], qkv[:, HQ + HKV:], ctx)
        d = self.rule(dqkv[:, :HK], dqkv[:, HK:2 * HK], dqkv[:, 2 * HK:], g, beta, ctx)
        y = self.lin(qkv[:, HQ:HQ + HKV], qkv[:, HQ:HQ + HKV], qkv[:, HQ + HKV:], ctx)
        logits = torch.cat([x.float().flatten(1) for x in (a, d, y)], 1) @ self.head * 0.1
        return a, d, y, logits

    def check(self, history, row, outputs=None):
        """What row `row` has cached, and (last token's) outputs, against a history of tokens."""
        n = len(history)
        t = torch.tensor(history)
        qkv, dqkv = self.qkv[t], self.dqkv[t]
        q, k, v = qkv[:, :HQ], qkv[:, HQ:HQ + HKV], qkv[:, HQ + HKV:]
        pages = self.pool.page_table[row].tolist()
        assert self.pool.seq_lens[row].item() == n
        at = [pages[p // BS] * BS + p % BS for p in range(n)]
        flat = lambda x: x.view(-1, HKV, D)[at].cpu()  # noqa: E731
        assert torch.equal(flat(self.att.k_cache), k) and torch.equal(flat(self.att.v_cache), v)
        assert torch.equal(flat(self.att.v16_cache), (v.float() / 16).to(torch.float16))
        ref, finals, reach = delta(dqkv[:, :HK], dqkv[:, HK:2 * HK], dqkv[:, 2 * HK:], self.g[t], self.beta[t], [0, n],
                                   D ** -0.5, [None], 1e-6)
        S, E = finals[0]
        err = (self.rule.state_cache[row].double().cpu() - S).abs()
        assert (err <= 128 * 2.0 ** -24 * E[..., None] + 1e-30).all()
        lref, lfinals, lweight = linear(k, k, v, self.decay, [0, n], D ** -0.5, [None])
        S, A = lfinals[0]
        assert ((self.lin.state_cache[row].double().cpu() - S).abs() <= 2.0 ** -13 * A).all()
        if outputs is not None:
            a, d, y = (x.double().cpu() for x in outputs)
            i32 = lambda *z: np.asarray(z, dtype=np.int32)  # noqa: E731
            want, _ = oracle.attn_varlen(q[-1:], k, v, i32(0, 1), i32(0, n), HQ, HKV, D, D ** -0.5, True)
            assert_close(a[None], want.reshape(1, HQ, D), "attention")
            rm, re = reach
            assert ((d - ref[-1]).abs() <= 2.0 ** -8 * ref[-1].abs() + 2.0 ** -14 * rm[-1]
                    + 128 * 2.0 ** -24 * re[-1] + 1e-30).all()
            assert ((y - lref[-1]).abs() <= 2.0 ** -8 * lref[-1].abs() + 2.0 ** -13 * lweight[-1]).all()


@pytest.mark.parametrize("R,W,steps", [(1, 1, 3), (2, 3, 9), (3, 4, 6)])
def test_a_search_over_attention_and_delta_layers(R, W, steps):
    gen = torch.Generator().manual_seed(R * 10 + W)
    rows = torch.randperm(R * W + 2, generator=gen)[:R * W].to(torch.int32).view(R, W)
    m = _Model(R * W + 2)
    prompts = [torch.randint(0, VOCAB, (n,), generator=gen).tolist() for n in (21, 40, 5)[:R]]
    lens = torch.tensor([len(p) for p in prompts], dtype=torch.int32, device="cuda")
    beams = Beams(m.pool, rows.cuda())
    av.get_last_device_error()
    # the prompts run in the first beams; the others' rows grow by as much
    firsts = beams.rows[:, 0].contiguous()
    total = sum(map(len, prompts))
    ctx = m.pool.context(m.pool.grow(lens, total, request_rows=firsts), True, max(map(len, prompts)), BS * M,
                         state_slots=firsts)
    tokens = torch.tensor(sum(prompts, []), dtype=torch.int32, device="cuda")
    out = m.run(tokens, ctx)
    if W > 1:
        others = beams.rows[:, 1:].contiguous().view(-1)
        m.pool.grow(lens.repeat_interleave(W - 1), total * (W - 1), request_rows=others)
    beams.start(m.layers)
    last = torch.tensor(np.cumsum([len(p) for p in prompts]) - 1, device="cuda")
    logits = out[3][last].repeat_interleave(W, 0).contiguous()           # the first beam's count, the others' do not
    history = [[list(p) for _ in range(W)] for p in prompts]
    scores = torch.full((R, W), float("-inf"))
    scores[:, 0] = 0
    for r in range(R):
        for w in range(W):
            m.check(history[r][w], int(beams.rows[r, w]))
    for step in range(steps):
        tokens, parents, new = beams.select(logits)
        want = select(logits.cpu(), scores.view(-1), W, W)
        assert torch.equal(tokens.cpu(), want[0]) and torch.equal(parents.cpu(), want[1])
        scores = new.cpu()
        beams.advance(parents, new, m.layers)
        history = [[history[r][int(p)] + [int(t)] for p, t in zip(parents[r], tokens[r])] for r in range(R)]
        assert sorted(beams.rows.view(-1).tolist()) == sorted(rows.view(-1).tolist())
        flat = beams.rows.view(-1)
        ones = torch.ones(R * W, dtype=torch.int32, device="cuda")
        t = m.pool.grow(ones, R * W, request_rows=flat)
        ctx = m.pool.context(t, False, 1, BS * M, state_slots=flat)
        out = m.run(tokens.view(-1), ctx)
        logits = out[3]
        for r in range(R):
            for w in range(W):
                i = r * W + w
                m.check(history[r][w], int(flat[i]), tuple(x[i] for x in out[:3]))
    assert av.get_last_device_error()[0] == 0


def test_one_search_step_captured_and_replayed():
    """Selection, rows and copies as one graph, replayed on other logits."""
    R, W, gen = 2, 4, torch.Generator().manual_seed(3)
    m = _Model(R * W)
    beams = Beams(m.pool, torch.arange(R * W, dtype=torch.int32, device="cuda").view(R, W))
    m.pool.grow(torch.full((R * W,), 20, dtype=torch.int32, device="cuda"), 20 * R * W)
    for c in (m.att.k_cache, m.att.v_cache, m.att.v16_cache, m.rule.state_cache, m.lin.state_cache):
        c.copy_(torch.randn(c.shape, generator=gen).to(c.dtype))
    beams.scores.copy_(-torch.rand(R, W, generator=gen))
    caches = [m.att.k_cache, m.att.v_cache, m.att.v16_cache, m.rule.state_cache, m.lin.state_cache]
    start = [c.clone() for c in caches]
    logits = torch.randn(R * W, VOCAB, generator=gen).cuda()

    def step():
        rows, scores = beams.rows, beams.scores
        tokens, parents, new = beams.select(logits)
        beams.advance(parents, new, m.layers)
        got = beams.rows, tokens, new
        beams.rows, beams.scores = rows, scores
        return got

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            got = step()
    side.synchronize()
    for _ in range(3):
        logits.copy_(torch.randn(R * W, VOCAB, generator=gen))
        for c, x in zip(caches, start):
            c.copy_(x)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        have = [x.clone() for x in got] + [c.clone() for c in caches]
        for c, x in zip(caches, start):
            c.copy_(x)
        want = list(step()) + caches
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(have, want))
    assert av.get_last_device_error()[0] == 0
