"""The delta-rule and beam-search entries on a machine without a GPU: refusals on the host."""
import ctypes

import pytest
import torch

import attention_attn_varlen_gb300 as av
import attention_attn_varlen_gb300.attention as at

# accepted calls below carry made-up addresses: they must find no device to run on
needs_no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="passes made-up device addresses")

FAKE = ctypes.c_void_p(0x1000)
ODD = ctypes.c_void_p(0x1008)


@pytest.fixture(scope="module")
def L():
    av.build()
    return av.lib()


@needs_no_gpu
def test_delta_refusals(L):
    def call(B=2, T=10, Hk=2, Hv=4, D=64, scale=0.1, eps=-1.0, slots_n=4, state=FAKE, slots=FAKE, q=FAKE, cu=FAKE, qs=0,
             gs=0, bs=0, max_len=100, ws=FAKE, ws_bytes=1 << 40, g=FAKE, beta=FAKE):
        return L.attn_delta_fwd(q, FAKE, FAKE, FAKE, g, beta, cu, state, slots, None, None, B, T, max_len, Hk, Hv, D,
                                scale, eps, slots_n, qs, 0, 0, 0, gs, bs, ws, ws_bytes, None)

    assert call() == 7                                   # accepted: only the device is missing
    assert call(T=0) == 0 and call(max_len=0) == 0       # nothing to do
    assert call(B=0) == 1 and call(T=-1) == 1 and call(max_len=-1) == 1
    assert call(Hv=3) == 1 and call(Hk=0) == 1 and call(Hk=4, Hv=2) == 1
    assert call(D=96) == 2 and call(B=65536) == 2 and call(T=2 ** 31 - 1) == 2 and call(Hk=65536, Hv=65536) == 2
    assert call(B=65535, Hk=60000, Hv=60000) == 2        # more CTAs than a grid has
    assert call(q=None) == 1 and call(cu=None) == 1 and call(g=None) == 1 and call(beta=None) == 1
    assert call(scale=0.0) == 1 and call(scale=float("inf")) == 1 and call(eps=float("nan")) == 1
    assert call(eps=0.0) == 7 and call(eps=1e-6) == 7
    assert call(state=None) == 1 and call(slots=None) == 1 and call(slots_n=0) == 1
    assert call(state=None, slots=None) == 7
    assert call(qs=2 * 64 + 4) == 1 and call(qs=64) == 1 and call(q=ODD) == 1 and call(state=ctypes.c_void_p(0x1004)) == 1
    assert call(gs=3) == 1 and call(bs=3) == 1 and call(gs=5, bs=9) == 7
    need = L.attn_delta_workspace_size(2, 10, 2, 4, 64, 100)
    if need:
        assert call(ws=None) == 1 and call(ws_bytes=need - 1) == 3 and call(ws=ctypes.c_void_p(0x1010)) == 1
        assert call(ws_bytes=need) == 7
    for bad in ((0, 10, 2, 4, 64, 100), (2, -1, 2, 4, 64, 100), (2, 10, 3, 4, 64, 100), (2, 10, 2, 4, 32, 100),
                (2, 10, 2, 4, 64, -1)):
        assert L.attn_delta_workspace_size(*bad) == 0

    def step(B=2, Hk=2, Hv=4, D=64, state=FAKE, slots=FAKE, vs=0):
        return L.attn_delta_decode(FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, state, slots, None, B, Hk, Hv, D, 0.1, -1.0, 4, 0,
                                   0, vs, 0, 0, 0, None)

    assert step() == 7 and step(state=None) == 1 and step(slots=None) == 1 and step(B=0) == 1 and step(D=32) == 2
    assert step(Hv=5) == 1 and step(vs=250) == 1 and step(vs=264) == 7


@needs_no_gpu
def test_beam_refusals(L):
    def call(R=2, W=4, V=1000, k=8, stride=0, dtype=1, x=FAKE, s=FAKE, t=FAKE, ws=FAKE, ws_bytes=1 << 40):
        return L.attn_beam_select(x, s, R, W, V, k, stride, dtype, t, FAKE, FAKE, ws, ws_bytes, None)

    assert call() == 7 and call(dtype=0) == 7 and call(stride=1001) == 7 and call(x=ctypes.c_void_p(0x1002)) == 7
    assert call(R=0) == 1 and call(W=0) == 1 and call(V=0) == 1 and call(k=0) == 1 and call(dtype=2) == 1
    assert call(stride=999) == 1 and call(x=None) == 1 and call(s=None) == 1 and call(t=None) == 1
    assert call(W=33) == 2 and call(k=33) == 2 and call(V=1 << 30) == 2 and call(R=1 << 23) == 2
    assert call(W=32, k=32) == 7
    assert call(ws=None) == 1 and call(ws=ODD) == 1
    need = L.attn_beam_select_workspace_size(2, 4, 1000, 8)
    assert need > 0 and call(ws_bytes=need - 1) == 3 and call(ws_bytes=need) == 7
    assert L.attn_beam_select_workspace_size(2, 33, 1000, 8) == 0

    rows = lambda R=2, W=4, p=FAKE, o=FAKE: L.attn_beam_rows(p, FAKE, o, FAKE, R, W, None)  # noqa: E731
    assert rows() == 7 and rows(R=0) == 1 and rows(W=0) == 1 and rows(W=33) == 2 and rows(p=None) == 1 and rows(o=None) == 1

    def copy(n=4, slots=8, size=64, c=FAKE, src=FAKE):
        return L.attn_copy_states(c, src, FAKE, n, slots, size, None)

    assert copy() == 7 and copy(n=0, c=None) == 0 and copy(n=-1) == 1 and copy(slots=0) == 1
    assert copy(size=0) == 1 and copy(size=24) == 1 and copy(c=None) == 1 and copy(c=ODD) == 1 and copy(src=None) == 1

    def pages(n=4, rows=8, M=5, bs=16, blocks=100, H=2, D=64, k=FAKE, table=FAKE, lens=FAKE):
        return L.attn_copy_kvcache(k, FAKE, None, FAKE, FAKE, n, table, lens, None, rows, M, bs, blocks, H, D, None)

    assert pages() == 7 and pages(n=0, k=None) == 0 and pages(n=-1) == 1 and pages(rows=0) == 1 and pages(M=0) == 1
    assert pages(bs=24) == 1 and pages(bs=8) == 1 and pages(blocks=0) == 1 and pages(H=0) == 1 and pages(D=0) == 1
    assert pages(k=None) == 1 and pages(table=None) == 1 and pages(lens=None) == 1
    assert pages(M=1 << 27) == 2 and pages(blocks=1 << 27) == 2


def test_the_binding_refuses_cpu_tensors():
    q = torch.zeros(2, 2, 64, dtype=torch.bfloat16)
    i32 = torch.zeros(2, dtype=torch.int32)
    g = torch.zeros(2, 2)
    with pytest.raises(ValueError, match="CUDA"):
        av.delta_attn_varlen_fwd(q, q, q, g, g, i32, 2)
    with pytest.raises(ValueError, match="CUDA"):
        av.delta_attn_decode(q, q, q, g, g, torch.zeros(2, 2, 64, 64), i32)
    with pytest.raises(ValueError, match="CUDA"):
        av.beam_select(torch.zeros(4, 10), torch.zeros(4), 2, 2)
    with pytest.raises(ValueError, match="CUDA"):
        av.beam_rows(i32.view(1, 2), i32.view(1, 2))
    with pytest.raises(ValueError, match="CUDA"):
        av.copy_states(torch.zeros(2, 4), i32, i32)
    with pytest.raises(ValueError, match="CUDA"):
        av.copy_kvcache(q[None], q[None], i32, i32, i32.view(1, 2), i32[:1])


def _i32(*x):
    return torch.tensor(x, dtype=torch.int32)


def test_the_delta_layer_goes_by_the_steps_tables(monkeypatch):
    """As LinearAttention: offsets where there are some, one row per sequence without
    them, and refusals where neither fits."""
    calls = []
    for name in ("delta_attn_decode", "delta_attn_varlen_fwd"):
        monkeypatch.setattr(at, name, lambda q, k, v, g, b, *a, name=name, **kw: (calls.append((name, a, kw)),
                                                                                  torch.zeros_like(v))[1])
    layer = at.DeltaAttention(1, 2, 64, 0.5, qk_norm_eps=None)

    def run(ctx, rows):
        calls.clear()
        x = torch.zeros(rows, 64)
        y = layer(x, x, torch.zeros(rows, 128), torch.zeros(rows, 2), torch.zeros(rows, 2), ctx)
        assert y.shape == (rows, 128)
        return calls[0]

    # a prompt without a cache starts from zero and keeps nothing
    name, a, kw = run(at.AttentionContext(True, cu_seqlens_q=_i32(0, 3, 5), max_seqlen_q=3), 5)
    assert name == "delta_attn_varlen_fwd" and a[0].tolist() == [0, 3, 5] and a[1:] == (3, 0.5)
    assert kw["state_cache"] is None and kw["state_slots"] is None and kw["qk_norm_eps"] is None
    with pytest.raises(ValueError, match="state cache"):
        run(at.AttentionContext(False, state_slots=_i32(0, 1)), 2)
    layer.state_cache = torch.zeros(4, 2, 64, 64)
    with pytest.raises(ValueError, match="state_slots"):
        run(at.AttentionContext(False), 2)
    name, a, kw = run(at.AttentionContext(False, state_slots=_i32(0, 1), past_lens=_i32(3, 0)), 2)
    assert name == "delta_attn_decode" and kw["context_lens"].tolist() == [3, 0]
    with pytest.raises(ValueError, match="offsets"):
        run(at.AttentionContext(False, state_slots=_i32(0, 1)), 4)
    with pytest.raises(ValueError, match="past_lens"):
        run(at.AttentionContext(False, state_slots=_i32(0, 1), cu_seqlens_q=_i32(0, 2, 4), max_seqlen_q=2), 4)
    name, a, kw = run(at.AttentionContext(False, state_slots=_i32(0, 1), cu_seqlens_q=_i32(0, 2, 4), max_seqlen_q=2,
                                          past_lens=_i32(9, 9), cache_seqlens=_i32(11, 9)), 4)
    assert name == "delta_attn_varlen_fwd" and a[1] == 2 and kw["cache_seqlens"].tolist() == [11, 9]
    with pytest.raises(ValueError, match="multiple"):
        at.DeltaAttention(2, 3, 64, 0.5)


def test_beams_hand_the_same_rows_to_every_cache(monkeypatch):
    calls = []
    monkeypatch.setattr(at, "beam_rows", lambda p, r: (r + 100, p))
    monkeypatch.setattr(at, "copy_kvcache", lambda *a, **kw: calls.append(("kv", a, kw)))
    monkeypatch.setattr(at, "copy_states", lambda *a: calls.append(("states", a, {})))
    pool = at.PagePool(8, 16, 6, 2, device="cpu")
    beams = at.Beams(pool, _i32(0, 1, 2, 3, 4, 5).view(2, 3))
    assert beams.scores.tolist() == [[0.0, -float("inf"), -float("inf")]] * 2
    att, rule = at.Attention(2, 64, 0.5, 1), at.DeltaAttention(1, 1, 64, 0.5)
    att.k_cache = att.v_cache = torch.zeros(8, 16, 1, 64)
    rule.state_cache = torch.zeros(6, 1, 64, 64)
    beams.start((att, rule))
    assert beams.scores[0, 0] == 0 and beams.first_tokens is not pool.seq_lens
    assert [c[0] for c in calls] == ["kv", "states"] and calls[0][2]["first_tokens"] is None
    calls.clear()
    new = torch.zeros(2, 3)
    beams.advance(_i32(0, 0, 1, 2, 2, 2).view(2, 3), new, (rule, att))
    assert beams.scores is new and [c[0] for c in calls] == ["states", "kv"]
    assert calls[0][1][2] is beams.rows and calls[1][2]["first_tokens"] is beams.first_tokens
    assert beams.rows.tolist() == [[200, 201, 202], [203, 204, 205]]
