"""One Beams object for one search after the other over the same request rows: the second
copies its whole prompts and begins from its first beams alone.  Checked as
a single search is, against every beam's own history (see test_gpu_beam_search)."""
import numpy as np
import pytest
import torch

import attention_attn_varlen_gb300 as av
import attention_attn_varlen_gb300.attention as at
from _delta_reference import select
from test_gpu_beam_search import BS, M, VOCAB, _Model


def _search(m, beams, prompts, steps):
    R, W = beams.rows.shape
    lens = torch.tensor([len(p) for p in prompts], dtype=torch.int32, device="cuda")
    total = sum(map(len, prompts))
    firsts = beams.rows[:, 0].contiguous()
    ctx = m.pool.context(m.pool.grow(lens, total, request_rows=firsts), True, max(map(len, prompts)), BS * M,
                         state_slots=firsts)
    out = m.run(torch.tensor(sum(prompts, []), dtype=torch.int32, device="cuda"), ctx)
    others = beams.rows[:, 1:].contiguous().view(-1)
    m.pool.grow(lens.repeat_interleave(W - 1), total * (W - 1), request_rows=others)
    beams.start(m.layers)
    logits = out[3][torch.tensor(np.cumsum([len(p) for p in prompts]) - 1, device="cuda")].repeat_interleave(W, 0)
    history = [[list(p) for _ in range(W)] for p in prompts]
    scores = torch.full((R, W), float("-inf"))
    scores[:, 0] = 0
    for r in range(R):
        for w in range(W):
            m.check(history[r][w], int(beams.rows[r, w]))
    for _ in range(steps):
        tokens, parents, new = beams.select(logits.contiguous())
        want = select(logits.cpu(), scores.view(-1), W, W)
        assert torch.equal(tokens.cpu(), want[0]) and torch.equal(parents.cpu(), want[1])
        scores = new.cpu()
        beams.advance(parents, new, m.layers)
        history = [[history[r][int(p)] + [int(t)] for p, t in zip(parents[r], tokens[r])] for r in range(R)]
        flat = beams.rows.view(-1)
        t = m.pool.grow(torch.ones_like(flat), R * W, request_rows=flat)
        out = m.run(tokens.view(-1), m.pool.context(t, False, 1, BS * M, state_slots=flat))
        logits = out[3]
        for r in range(R):
            for w in range(W):
                m.check(history[r][w], int(flat[r * W + w]), tuple(x[r * W + w] for x in out[:3]))


@pytest.mark.gpu
def test_one_search_after_the_other():
    R, W, gen = 2, 3, torch.Generator().manual_seed(5)
    m = _Model(R * W)
    beams = at.Beams(m.pool, torch.randperm(R * W, generator=gen).to(torch.int32).view(R, W).cuda())
    av.get_last_device_error()
    for lens in ([50, 21], [9, 40], [1, 70]):
        prompts = [torch.randint(0, VOCAB, (n,), generator=gen).tolist() for n in lens]
        _search(m, beams, prompts, 4)
        flat = beams.rows.view(-1)
        m.pool.trim(torch.zeros_like(flat), request_rows=flat)
    assert av.get_last_device_error()[0] == 0


def test_a_second_start_forgets_the_first_search(monkeypatch):
    calls = []
    monkeypatch.setattr(at, "beam_rows", lambda p, r: (r, p))
    monkeypatch.setattr(at, "copy_kvcache", lambda *a, **kw: calls.append(kw["first_tokens"]))
    pool = at.PagePool(8, 16, 4, 2, device="cpu")
    beams = at.Beams(pool, torch.arange(4, dtype=torch.int32).view(2, 2))
    att = at.Attention(2, 64, 0.5, 1)
    att.k_cache = att.v_cache = torch.zeros(8, 16, 1, 64)
    pool.seq_lens.fill_(7)
    beams.start((att,))
    beams.advance(torch.zeros(2, 2, dtype=torch.int32), torch.tensor([[-1.0, -2.0], [-3.0, -4.0]]), (att,))
    assert calls[0] is None and calls[1].tolist() == [7] * 4
    pool.seq_lens.fill_(5)
    beams.start((att,))
    assert calls[2] is None and beams.first_tokens.tolist() == [5] * 4
    assert beams.scores.tolist() == [[0.0, -float("inf")]] * 2
    # a first search's own scores stay as its caller set them
    beams = at.Beams(pool, torch.arange(4, dtype=torch.int32).view(2, 2))
    beams.scores[:, 1] = -1.0
    beams.start()
    assert beams.scores.tolist() == [[0.0, -1.0]] * 2
