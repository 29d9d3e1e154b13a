"""A model's serving steps on the GPU, as a program runs them: the page pool grows
and builds the step's tables, an attention layer with rotary positions stores and
attends, a linear-attention layer advances its states; prompts, decode steps,
speculative tokens that are taken back, a request that ends and one that takes its
pages.  Every step against 64-bit references over the whole history."""
import numpy as np
import pytest
import torch

import attention_attn_varlen_gb300 as av
import oracle
from attention_attn_varlen_gb300.attention import Attention, LinearAttention, PagePool, Rotary
from _step_reference import linear, rope
from _util import assert_close

pytestmark = pytest.mark.gpu

Hq, Hkv, D, BS, R = 8, 2, 128, 16, 4


@pytest.mark.parametrize("axes", [1, 3])
def test_serving_steps(axes):
    gen = torch.Generator().manual_seed(5)
    pool = PagePool(60, BS, R, 30)
    inv = (10000.0 ** (-torch.arange(D // 2, dtype=torch.float64) / (D // 2))).float()
    axis = None if axes == 1 else bytes([i % axes for i in range(D // 2)])
    g = torch.tensor([-0.3, -0.01])
    att = Attention(Hq, D, D ** -0.5, Hkv, rotary=Rotary(inv.cuda(), axis))
    att.k_cache = torch.full((60, BS, Hkv, D), float("nan"), dtype=torch.bfloat16, device="cuda")
    att.v_cache = torch.full_like(att.k_cache, float("nan"))
    lin = LinearAttention(Hq, D, D ** -0.5, Hkv, g.cuda())
    lin.state_cache = torch.full((R, Hkv, D, D), float("nan"), device="cuda")
    empty = lambda h: torch.empty(0, h, D, dtype=torch.bfloat16)  # noqa: E731
    hist = {r: [empty(Hkv), empty(Hkv), empty(Hkv)] for r in range(R)}       # rotated k, raw k, v of each request
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    av.get_last_device_error()

    def step(rows, new, kind, pad=0):
        """Run both layers on a step and check them; returns the step's tables."""
        n = sum(new)
        mk = lambda h: torch.randn(n + pad, h, D, generator=gen).to(torch.bfloat16)  # noqa: E731
        q, k, v = mk(Hq), mk(Hkv), mk(Hkv)
        past = [len(hist[r][0]) for r in rows]
        t = pool.grow(i32(new), n + pad, request_rows=i32(rows))
        pos = t.positions if axes == 1 else torch.stack([t.positions, t.positions // 7, t.positions % 5])
        ctx = pool.context(t, kind != "decode", max(new), max(p + m for p, m in zip(past, new)),
                           paged=kind != "prompt", state_slots=i32(rows), positions=pos)
        lin_state_old = lin.state_cache.clone()
        o = att(q.cuda(), k.cuda(), v.cuda(), ctx).cpu()
        y = lin(q.cuda(), k.cuda(), v.cuda(), ctx).cpu()
        torch.cuda.synchronize()
        assert t.context_lens.tolist() == past
        cu = np.concatenate([[0], np.cumsum(new)])
        p = np.concatenate([np.arange(a, a + m) for a, m in zip(past, new)])
        pos3 = torch.tensor(np.stack([p, p // 7, p % 5])[:axes])
        q_rot = rope(q[:n], pos3, inv, axis, False, 1.0).to(torch.bfloat16)
        k_rot = rope(k[:n], pos3, inv, axis, False, 1.0).to(torch.bfloat16)
        for b, r in enumerate(rows):
            for x, y_new in zip(range(3), (k_rot, k, v)):
                hist[r][x] = torch.cat([hist[r][x], y_new[cu[b]:cu[b + 1]]])
        lens = [len(hist[r][0]) for r in rows]
        cu_k = np.concatenate([[0], np.cumsum(lens)])
        i32n = lambda x: np.asarray(x, dtype=np.int32)  # noqa: E731
        ref, _ = oracle.attn_varlen(q_rot, torch.cat([hist[r][0] for r in rows]), torch.cat([hist[r][2] for r in rows]),
                                    i32n(cu), i32n(cu_k), Hq, Hkv, D, D ** -0.5, True)
        assert_close(o[:n], ref.reshape(n, Hq, D), kind)
        starts = [lin_state_old[r].double().cpu() if a else None for r, a in zip(rows, past)]
        lref, finals, weight = linear(q[:n], k[:n], v[:n], g, cu, D ** -0.5, starts)
        err = (y[:n].double() - lref).abs()
        assert (err <= 2.0 ** -8 * lref.abs() + 2.0 ** -13 * weight).all(), kind
        for b, r in enumerate(rows):
            e = (lin.state_cache[r].double().cpu() - finals[b][0]).abs()
            assert (e <= 2.0 ** -13 * finals[b][1] + 1e-30).all(), kind
        return t

    step([0, 2, 3], [37, 130, 5], "prompt")
    step([0, 2, 3], [1, 1, 1], "decode")
    step([3, 0], [1, 1], "decode")                       # another set of requests, in another order
    step([0, 2], [40, 3], "prefix")                      # a prompt's next piece
    # speculative tokens: both layers run over them, then the pool and the states go back
    kept = lin.state_cache.clone()
    t = pool.grow(i32([9, 20]), 29, request_rows=i32([2, 0]))
    free = pool.num_free.item()
    pool.trim(t.context_lens, request_rows=i32([2, 0]))
    assert pool.num_free.item() >= free and pool.seq_lens.tolist() == [len(hist[r][0]) for r in range(R)]
    assert torch.equal(kept.nan_to_num(), lin.state_cache.nan_to_num())
    step([0, 2, 3], [1, 1, 1], "decode")
    # request 2 ends; a new one takes its row, its pages and its state slot
    before = pool.num_free.item()
    pool.trim(i32([0]), request_rows=i32([2]))
    assert pool.num_free.item() == before + -(-len(hist[2][0]) // BS)
    hist[2] = [empty(Hkv), empty(Hkv), empty(Hkv)]
    step([2, 1], [33, 64], "prompt")
    step([0, 1, 2, 3], [1, 1, 1, 1], "decode")
    assert av.get_last_device_error()[0] == 0


def test_a_captured_step_is_the_eager_one():
    """Tables, rotary store, attention and linear attention of a decode step in one graph,
    replayed while the requests grow, with a padded batch entry: the bits of eager steps."""
    gen = torch.Generator(device="cuda").manual_seed(9)
    rnd = lambda *s: torch.randn(*s, generator=gen, device="cuda").bfloat16()  # noqa: E731
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    inv = torch.rand(D // 2, generator=gen, device="cuda")
    g = torch.tensor([-0.3, -0.01], device="cuda")
    rows, new, slots, start = i32([3, 0, 1, 2]), i32([1, 1, 1, 0]), i32([3, 0, 1, -1]), i32([40, BS - 2, 0, 0])

    def build():
        pool = PagePool(80, BS, R, 30)
        pool.grow(start, 200, request_rows=rows)
        att = Attention(Hq, D, D ** -0.5, Hkv, rotary=Rotary(inv))
        att.k_cache, att.v_cache = (torch.zeros(80, BS, Hkv, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        lin = LinearAttention(Hq, D, D ** -0.5, Hkv, g)
        lin.state_cache = torch.ones(R, Hkv, D, D, device="cuda")
        x = [torch.zeros(4, h, D, dtype=torch.bfloat16, device="cuda") for h in (Hq, Hkv, Hkv)]

        def step():
            t = pool.grow(new, 4, request_rows=rows)
            ctx = pool.context(t, False, 1, 30 * BS, state_slots=slots)
            return att(*x, ctx), lin(*x, ctx), t
        return pool, att, lin, x, step

    a, b = build(), build()
    torch.cuda.synchronize()
    keep = [t.clone() for t in (b[0].seq_lens, b[0].page_table, b[0].num_free, b[2].state_cache)]
    b[4]()                                               # once eagerly, then back to the start
    torch.cuda.synchronize()
    for t, old in zip((b[0].seq_lens, b[0].page_table, b[0].num_free, b[2].state_cache), keep):
        t.copy_(old)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = b[4]()
    av.get_last_device_error()
    for n in range(BS + 3):                              # past a page's end
        q = [rnd(*t.shape) for t in a[3]]
        for t, u, v in zip(a[3], b[3], q):
            t.copy_(v)
            u.copy_(v)
        want = a[4]()
        graph.replay()
        assert torch.equal(got[0][:3], want[0][:3]) and torch.equal(got[1][:3], want[1][:3])
        assert all(torch.equal(x, y) for x, y in zip(got[2], want[2]))
    assert torch.equal(a[2].state_cache, b[2].state_cache) and torch.equal(a[1].k_cache, b[1].k_cache)
    assert a[0].seq_lens.tolist()[:4] == b[0].seq_lens.tolist()[:4] == [BS - 2 + BS + 3, BS + 3, 0, 40 + BS + 3]
    assert av.get_last_device_error()[0] == 0
