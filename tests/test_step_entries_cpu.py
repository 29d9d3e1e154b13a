"""The serving-step entries on a machine without a GPU: refusals on the host, and
the layers' routing."""
import ctypes

import pytest
import torch

import attention_attn_varlen_gb300 as av
import attention_attn_varlen_gb300.attention as at

# accepted calls below carry made-up addresses: they must find no device to run on
needs_no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="passes made-up device addresses")


@pytest.fixture(scope="module")
def L():
    av.build()
    return av.lib()


FAKE = ctypes.c_void_p(0x1000)


@needs_no_gpu
def test_step_tables_refusals(L):
    def call(B=4, R=8, M=16, bs=16, pages=100, T=64, rows=FAKE, ws=FAKE, ws_bytes=1 << 20, lens=FAKE, slots=FAKE,
             bt=FAKE):
        return L.attn_step_tables(rows, lens, FAKE, FAKE, FAKE, FAKE, B, R, M, bs, pages, T, bt, slots, FAKE, FAKE,
                                  FAKE, FAKE, FAKE, ws, ws_bytes, None)

    assert call() == 7                                   # accepted: only the device is missing
    assert call(lens=None) == 1 and call(slots=None) == 1 and call(bt=None) == 1
    assert call(slots=None, T=0) == 7                    # no tokens: nothing to point at
    assert call(B=0) == 1 and call(R=0) == 1 and call(M=0) == 1 and call(pages=0) == 1 and call(T=-1) == 1
    assert call(bs=24) == 1 and call(bs=8) == 1
    assert call(rows=None, B=9) == 1                     # entry b is row b: more entries than rows
    assert call(rows=None, B=8) == 7
    assert call(ws=None) == 1 and call(ws=ctypes.c_void_p(0x1004)) == 1
    assert call(ws_bytes=4 * 20 - 1) == 3
    assert call(B=65536, R=65536) == 2
    assert call(M=1 << 27) == 2 and call(pages=1 << 27) == 2 and call(T=2 ** 31 - 1) == 2
    assert L.attn_step_tables_workspace_size(4) == 80
    assert L.attn_step_tables_workspace_size(0) == 0 and L.attn_step_tables_workspace_size(65536) == 0

    def trim(B=4, bs=16, ws_bytes=1 << 20, lens=FAKE):
        return L.attn_trim_pages(None, lens, FAKE, FAKE, FAKE, FAKE, B, 8, 16, bs, 100, FAKE, ws_bytes, None)

    assert trim() == 7 and trim(B=0) == 1 and trim(bs=17) == 1 and trim(lens=None) == 1 and trim(ws_bytes=0) == 3


@needs_no_gpu
def test_rope_store_refusals(L):
    def call(N=4, Hq=8, Hkv=2, D=128, rot=128, axes=1, axis=None, axis_stride=4, scale=1.0, q=FAKE, v=FAKE, q_out=FAKE,
             k_out=None, kc=FAKE, vc=FAKE, v16=None, slots=FAKE, qs=0, pos=FAKE):
        return L.attn_rope_store_kvcache(q, FAKE, v, pos, FAKE, axis, axes, axis_stride, rot, 0, scale, q_out, k_out,
                                         kc, vc, v16, slots, N, Hq, Hkv, D, qs, 0, 0, 0, 0, 64, None)

    assert call() == 7
    assert call(N=0, q=None) == 0                        # nothing to do
    assert call(N=-1) == 1 and call(Hq=0) == 1 and call(D=0) == 1 and call(D=7, rot=6) == 1
    assert call(rot=0) == 1 and call(rot=3) == 1 and call(rot=130) == 1
    assert call(D=512, rot=258) == 2 and call(D=512, rot=256) == 7
    assert call(scale=0.0) == 1 and call(scale=float("nan")) == 1 and call(scale=-1.0) == 1
    assert call(q=None) == 1 and call(pos=None) == 1 and call(q_out=None) == 1
    assert call(axes=3) == 1 and call(axes=0) == 1 and call(axes=5, axis=bytes(64)) == 2
    assert call(axes=3, axis=bytes(64)) == 7 and call(axes=3, axis=bytes(64), axis_stride=3) == 1
    assert call(axes=3, axis=bytes([3] * 64)) == 1       # an axis that does not exist
    assert call(kc=None) == 1 and call(vc=None) == 1 and call(slots=None) == 1 and call(v=None) == 1
    assert call(kc=None, vc=None, slots=None, v=None) == 1                   # the rotated k would go nowhere
    assert call(kc=None, vc=None, slots=None, v=None, k_out=FAKE) == 7
    assert call(kc=None, vc=None, slots=None, v16=FAKE, k_out=FAKE) == 1
    assert call(qs=100) == 1                             # rows overlap


@needs_no_gpu
def test_linear_refusals(L):
    def call(B=2, T=10, Hq=4, Hkv=2, D=64, scale=0.1, slots_n=4, state=FAKE, slots=FAKE, q=FAKE, cu=FAKE, qs=0,
             max_len=8, ws=FAKE, ws_bytes=1 << 40, g=FAKE):
        return L.attn_linear_varlen_fwd(q, FAKE, FAKE, FAKE, g, cu, state, slots, None, B, T, max_len, Hq, Hkv, D,
                                        scale, slots_n, qs, 0, 0, 0, ws, ws_bytes, None)

    assert call() == 7
    assert call(T=0) == 0 and call(B=0) == 1 and call(T=-1) == 1 and call(max_len=-1) == 1
    assert call(Hq=3) == 1 and call(D=96) == 2 and call(B=65536) == 2 and call(T=2 ** 31 - 1) == 2
    assert call(q=None) == 1 and call(cu=None) == 1 and call(g=None) == 1
    assert call(scale=0.0) == 1 and call(scale=float("inf")) == 1
    assert call(state=None) == 1 and call(slots=None) == 1 and call(slots_n=0) == 1
    assert call(state=None, slots=None) == 7
    assert call(qs=4 * 64 + 4) == 1 and call(q=ctypes.c_void_p(0x1008)) == 1 and call(state=ctypes.c_void_p(0x1004)) == 1

    def step(B=2, Hq=4, Hkv=2, D=64, state=FAKE, slots=FAKE):
        return L.attn_linear_decode(FAKE, FAKE, FAKE, FAKE, FAKE, state, slots, None, B, Hq, Hkv, D, 0.1, 4, 0, 0, 0,
                                    0, None)

    assert step() == 7 and step(state=None) == 1 and step(slots=None) == 1 and step(B=0) == 1 and step(D=32) == 2
    assert step(Hq=6, Hkv=4) == 1


def test_capacity_status_has_a_text(L):
    assert b"page" in L.attn_status_string(9)
    assert "page" in str(av.AttnError(9, "x"))


def test_the_binding_refuses_cpu_tensors_and_wrong_types():
    q = torch.zeros(2, 2, 64, dtype=torch.bfloat16)
    i32 = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        av.rope_store_kvcache(q, q, None, i32, torch.zeros(32))
    with pytest.raises(ValueError, match="CUDA"):
        av.linear_attn_decode(q, q, q, torch.zeros(2), torch.zeros(2, 2, 64, 64), i32)
    with pytest.raises(ValueError, match="CUDA"):
        av.step_tables(None, i32, i32, torch.zeros(2, 2, dtype=torch.int32), i32, i32[:1], 16, 4)


@pytest.fixture
def calls(monkeypatch):
    log = []

    def note(name, result=None):
        def f(*a, **kw):
            log.append((name, a, kw))
            return result(*a, **kw) if result else None
        return f

    def rope(q, k, *a, return_k=False, **kw):
        return (q + 1, k + 1) if return_k else q + 1

    monkeypatch.setattr(at, "rope_store_kvcache", note("rope", rope))
    monkeypatch.setattr(at, "store_kvcache", note("store"))
    for name in ("attn_varlen_fwd", "attn_decode_paged", "linear_attn_decode", "linear_attn_varlen_fwd"):
        monkeypatch.setattr(at, name, note(name, lambda q, *a, **kw: torch.zeros_like(q)))
    return log


def _ctx(prefill, n, **kw):
    cu = torch.tensor([0, n])
    return at.AttentionContext(prefill, slot_mapping=torch.arange(n), cu_seqlens_q=cu, cu_seqlens_k=cu, max_seqlen_q=n,
                               max_seqlen_k=n, positions=torch.arange(n), **kw)


def test_a_rotary_layer_rotates_and_stores_in_one_call(calls):
    layer = at.Attention(4, 16, 0.25, 2, rotary=at.Rotary(torch.ones(8), bytes(8), True, 1.5))
    q, k, v = torch.zeros(3, 64), torch.zeros(3, 32), torch.zeros(3, 32)
    layer(q, k, v, _ctx(True, 3))                        # no cache: only q and k, both used rotated
    (_, a, kw), (name, b, _) = calls
    assert a[2] is None and kw["return_k"] and kw["interleaved"] and kw["scale"] == 1.5 and kw["pair_axis"] == bytes(8)
    assert name == "attn_varlen_fwd" and b[0].eq(1).all() and b[1].eq(1).all() and b[2].eq(0).all()
    layer.k_cache = layer.v_cache = torch.zeros(4, 16, 2, 16)
    calls.clear()
    layer(q, k, v, _ctx(True, 3))                        # fresh prompts: attention reads the rotated k
    assert [c[0] for c in calls] == ["rope", "attn_varlen_fwd"] and calls[0][2]["return_k"]
    assert calls[0][1][5] is layer.k_cache and calls[1][1][1].eq(1).all()
    calls.clear()
    bt = torch.zeros(1, 2, dtype=torch.int32)
    layer(q, k, v, _ctx(True, 3, block_tables=bt))       # through the cache: k goes there only
    assert [c[0] for c in calls] == ["rope", "attn_varlen_fwd"] and not calls[0][2]["return_k"]
    assert calls[1][1][1] is layer.k_cache
    calls.clear()
    layer(q, k, v, _ctx(False, 3, block_tables=bt, context_lens=torch.ones(3, dtype=torch.int32)))
    assert [c[0] for c in calls] == ["rope", "attn_decode_paged"] and calls[1][1][0].eq(1).all()
    ctx = _ctx(True, 3)
    ctx.positions = None
    with pytest.raises(ValueError, match="positions"):
        layer(q, k, v, ctx)


def test_linear_layer_routes_by_step(calls):
    layer = at.LinearAttention(4, 64, 0.5, 2, torch.zeros(2))
    q, k, v = torch.zeros(3, 256), torch.zeros(3, 128), torch.zeros(3, 128)
    layer(q, k, v, _ctx(True, 3))
    assert calls[0][0] == "linear_attn_varlen_fwd" and calls[0][2]["state_cache"] is None
    with pytest.raises(ValueError):
        layer(q, k, v, _ctx(False, 3))
    layer.state_cache = torch.zeros(5, 2, 64, 64)
    with pytest.raises(ValueError, match="state_slots"):
        layer(q, k, v, _ctx(True, 3))
    calls.clear()
    slots, past = torch.arange(3, dtype=torch.int32), torch.ones(3, dtype=torch.int32)
    assert layer(q, k, v, _ctx(False, 3, state_slots=slots, past_lens=past)).shape == q.shape
    assert calls[0][0] == "linear_attn_decode" and calls[0][1][5] is slots and calls[0][2]["context_lens"] is past
    calls.clear()
    one = torch.zeros(1, dtype=torch.int32)
    layer(q, k, v, _ctx(False, 3, state_slots=one, past_lens=one))           # three tokens of one sequence
    assert calls[0][0] == "linear_attn_varlen_fwd" and calls[0][2]["context_lens"] is one
    with pytest.raises(ValueError, match="past_lens"):
        layer(q, k, v, _ctx(False, 3, state_slots=one))
    with pytest.raises(ValueError):
        at.LinearAttention(3, 64, 0.5, 2, torch.zeros(2))
