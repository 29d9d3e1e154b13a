"""The gated delta rule, the beam selection and the copies where sizes, offsets and
streams are unusual: offsets past 32 bits, the most sequences, rows and pairs,
streams of their own, workspaces that graphs share.  Everything is compared bit for bit
with the same work in an ordinary form."""
import pytest
import torch

import attention_attn_varlen_gb300 as av
from _step_reference import cu_of

pytestmark = pytest.mark.gpu


def i32(*x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _inputs(T, Hk, Hv, D, seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    q, k = (torch.randn(T, Hk, D, generator=gen, device="cuda").bfloat16() for _ in range(2))
    v = torch.randn(T, Hv, D, generator=gen, device="cuda").bfloat16()
    g, beta = (torch.rand(T, Hv, generator=gen, device="cuda") for _ in range(2))
    return q, k, v, -0.2 * g, beta


def _wide(x, stride):
    """The same rows, `stride` elements apart (only they are written)."""
    out = torch.empty(x.shape[0] * stride, dtype=x.dtype, device="cuda").as_strided(x.shape, (stride, *x.stride()[1:]))
    out.copy_(x)
    return out


@pytest.mark.parametrize("T", [1, 9, 130])
def test_states_past_32_bits(T):
    Hk, Hv, D, slots = 4, 32, 128, 4200                     # 2^19 elements a slot: 2.2e9 in all
    dev = _inputs(T, Hk, Hv, D)
    big = torch.empty(slots, Hv, D, D, device="cuda")
    small = torch.randn(1, Hv, D, D, device="cuda")
    big[slots - 1] = small[0]
    kw = dict(context_lens=i32(3), qk_norm_eps=1e-6)
    if T == 1:
        want = av.delta_attn_decode(*dev, small, i32(0), **kw)
        got = av.delta_attn_decode(*dev, big, i32(slots - 1), **kw)
    else:
        want = av.delta_attn_varlen_fwd(*dev, i32(0, T), T, state_cache=small, state_slots=i32(0), **kw)
        got = av.delta_attn_varlen_fwd(*dev, i32(0, T), T, state_cache=big, state_slots=i32(slots - 1), **kw)
    assert torch.equal(got, want) and torch.equal(big[slots - 1], small[0])
    av.copy_states(big, i32(slots - 1), i32(slots - 2))
    av.copy_states(big, i32(slots - 2), i32(0))
    assert torch.equal(big[slots - 2], small[0]) and torch.equal(big[0], small[0])
    assert av.get_last_device_error()[0] == 0


@pytest.mark.parametrize("lens", [[1] * 2200, [4] * 550, [2200], [100] * 22])
def test_rows_past_32_bits(lens):
    Hk, Hv, D, T, far = 2, 2, 64, 2200, 1 << 20             # row 2,199 starts at element 2.3e9
    dev = _inputs(T, Hk, Hv, D)
    cu, n, B = cu_of(lens).cuda(), max(lens), len(lens)
    wide = tuple(_wide(x, far) for x in dev[:3]) + tuple(_wide(x, far) for x in dev[3:])
    out = torch.empty(T * far, dtype=torch.bfloat16, device="cuda").as_strided((T, Hv, D), (far, D, 1))
    states = [torch.zeros(B, Hv, D, D, device="cuda") for _ in range(2)]
    slots = torch.arange(B, dtype=torch.int32, device="cuda")
    if n == 1:
        want = av.delta_attn_decode(*dev, states[0], slots, qk_norm_eps=1e-6)
        av.delta_attn_decode(*wide, states[1], slots, qk_norm_eps=1e-6, out=out)
    else:
        want = av.delta_attn_varlen_fwd(*dev, cu, n, state_cache=states[0], state_slots=slots, qk_norm_eps=1e-6)
        av.delta_attn_varlen_fwd(*wide, cu, n, state_cache=states[1], state_slots=slots, qk_norm_eps=1e-6, out=out)
    assert torch.equal(out, want) and torch.equal(*states)
    assert av.get_last_device_error()[0] == 0


@pytest.mark.parametrize("n", [1, 3, 17])
def test_as_many_sequences_as_there_can_be(n):
    """65,535 sequences; their bits do not depend on the company."""
    B, H, D = 65535, 1, 64
    lens = torch.full((B,), n)
    if n > 1:
        lens[::5] -= 1
        lens[7::1000] = 0
    cu = torch.nn.functional.pad(lens.cumsum(0), (1, 0)).to(torch.int32)
    T = int(cu[-1])
    dev = _inputs(T, H, H, D)
    state = torch.zeros(B, H, D, D, device="cuda")
    slots = torch.arange(B, dtype=torch.int32, device="cuda").flip(0)
    if n == 1:
        out = av.delta_attn_decode(*dev, state, slots, qk_norm_eps=1e-6)
    else:
        out = av.delta_attn_varlen_fwd(*dev, cu.cuda(), n, state_cache=state, state_slots=slots, qk_norm_eps=1e-6)
    for lo, hi in ((0, 100), (32000, 32100), (B - 100, B)):
        a, b = int(cu[lo]), int(cu[hi])
        part = [x[a:b] for x in dev]
        s = torch.zeros(hi - lo, H, D, D, device="cuda")
        at = torch.arange(hi - lo, dtype=torch.int32, device="cuda")
        if n == 1:
            want = av.delta_attn_decode(*part, s, at, qk_norm_eps=1e-6)
        else:
            want = av.delta_attn_varlen_fwd(*part, (cu[lo:hi + 1] - a).cuda(), n, state_cache=s, state_slots=at,
                                            qk_norm_eps=1e-6)
        assert torch.equal(out[a:b], want) and torch.equal(state[slots[lo:hi].long()], s)
    assert av.get_last_device_error()[0] == 0


@pytest.mark.parametrize("lens", [[5, 3, 16, 1], [70, 1, 200, 33]])
def test_a_padded_step_under_a_wide_bound(lens):
    """Rows and lengths up to a bound that a captured step takes: padded entries are empty, more rows
    than tokens."""
    Hk, Hv, D, T = 2, 4, 128, sum(lens)
    dev = _inputs(T + 300, Hk, Hv, D)
    B = len(lens)
    cu = cu_of(lens + [0, 0, 0]).cuda()
    s0, s1 = (torch.zeros(B + 1, Hv, D, D, device="cuda") for _ in range(2))
    slots = torch.tensor([*range(B), -1, -1, -1], dtype=torch.int32, device="cuda")
    out = torch.full((T + 300, Hv, D), 7.0, dtype=torch.bfloat16, device="cuda")
    av.delta_attn_varlen_fwd(*dev, cu, 4096, state_cache=s0, state_slots=slots, qk_norm_eps=1e-6, out=out)
    # the chunked form, whatever the lengths: as under its own bound
    want = av.delta_attn_varlen_fwd(*(x[:T] for x in dev), cu[:B + 1].contiguous(), max(max(lens), 17), state_cache=s1,
                                    state_slots=slots[:B].contiguous(), qk_norm_eps=1e-6)
    assert torch.equal(out[:T], want) and torch.equal(s0, s1) and out[T:].eq(7.0).all() and s0[B].eq(0).all()
    assert av.get_last_device_error()[0] == 0


def test_graphs_share_a_workspace():
    D, H = 64, 2
    runs = []
    sizes = [[2600], [100, 33, 0, 600], [40, 2561]]          # with and without segments
    ws = torch.empty(max(av.delta_attn_workspace_size(len(x), sum(x), H, H, D, max(x)) for x in sizes), dtype=torch.uint8,
                     device="cuda")
    for lens in sizes:
        dev, cu = _inputs(sum(lens), H, H, D, sum(lens)), cu_of(lens).cuda()
        want = av.delta_attn_varlen_fwd(*dev, cu, max(lens), qk_norm_eps=1e-6)
        out = torch.empty_like(want)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            av.delta_attn_varlen_fwd(*dev, cu, max(lens), qk_norm_eps=1e-6, out=out, workspace=ws)
        runs.append((graph, want, out, dev, cu))
    ws.fill_(0xA5)
    for _ in range(3):
        for graph, _, out, *_ in runs:
            out.zero_()
            graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(out, want) for _, want, out, *_ in runs)
    assert av.get_last_device_error()[0] == 0


def _make(name):
    gen = torch.Generator(device="cuda").manual_seed(3)
    if name == "select":
        x, s = torch.randn(24, 50000, generator=gen, device="cuda"), torch.zeros(24, device="cuda")
        return lambda stream: lambda: av.beam_select(x, s, 4, 8, stream=stream)
    if name == "rows":
        rows = torch.randperm(4096, generator=gen, device="cuda").int().view(512, 8)
        parents = torch.randint(0, 8, (512, 8), generator=gen, device="cuda").int()
        return lambda stream: lambda: av.beam_rows(parents, rows, stream=stream)
    lens = {"prompt": [200] * 3, "long": [4000], "few": [4] * 60, "step": [1] * 60}[name]
    dev, cu = _inputs(sum(lens), 4, 4, 64), cu_of(lens).cuda()
    state = torch.randn(len(lens), 4, 64, 64, generator=gen, device="cuda")
    slots, ones = torch.arange(len(lens), dtype=torch.int32, device="cuda"), torch.ones(len(lens), device="cuda").int()

    def make(stream):
        s = state.clone()
        torch.cuda.synchronize()
        if name == "step":
            return lambda: (av.delta_attn_decode(*dev, s, slots, qk_norm_eps=1e-6, stream=stream), s)
        return lambda: (av.delta_attn_varlen_fwd(*dev, cu, max(lens), state_cache=s, state_slots=slots, context_lens=ones,
                                                 qk_norm_eps=1e-6, stream=stream), s)
    return make


@pytest.mark.parametrize("name", ["prompt", "long", "few", "step", "select", "rows"])
def test_allocations_on_another_stream(name):
    make = _make(name)
    want = [x.clone() for x in make(None)()]
    side = torch.cuda.Stream()
    call = make(side)
    torch.cuda.empty_cache()
    # blocks of the outputs' and the workspace's sizes that the current stream frees while it is still to write them
    taken = [torch.empty_like(x) for x in want] + [torch.empty(n, dtype=torch.uint8, device="cuda")
                                                   for n in (512, 4096, 1 << 16, 1 << 18, 1 << 20, 1 << 21)]
    torch.cuda.synchronize()
    torch.cuda._sleep(200_000_000)                  # about 0.1 s
    for x in taken:
        x.view(torch.uint8).fill_(0xA5)
    del taken, x
    got = call()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert av.get_last_device_error()[0] == 0


def test_two_calls_at_once():
    """Prompts and a selection on streams of their own, workspaces of their own, many times over."""
    calls = [_make("long")(None), _make("prompt")(None)]
    want = [call()[0].clone() for call in calls] + list(_make("select")(None)())
    streams = [torch.cuda.Stream() for _ in range(3)]
    for _ in range(5):
        made = [_make("long")(streams[0]), _make("prompt")(streams[1]), _make("select")(streams[2])]
        torch.cuda.synchronize()
        got = [m() for m in made]
        torch.cuda.synchronize()
        got = [got[0][0], got[1][0], *got[2]]
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert av.get_last_device_error()[0] == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_logits_past_32_bits(dtype):
    R, W, V, k, far = 33, 4, 5000, 8, 1 << 24               # row 131 starts at element 2.2e9
    gen = torch.Generator(device="cuda").manual_seed(4)
    x = torch.randn(R * W, V, generator=gen, device="cuda").to(dtype)
    s = torch.randn(R * W, generator=gen, device="cuda")
    wide = torch.empty(R * W * far, dtype=dtype, device="cuda").as_strided((R * W, V), (far, 1))
    wide.copy_(x)
    assert all(torch.equal(a, b) for a, b in zip(av.beam_select(wide, s, W, k), av.beam_select(x, s, W, k)))


@pytest.mark.parametrize("R,W,V,k", [(70000, 1, 5, 3), (140000, 2, 3, 6), (300, 32, 2100, 32), (1, 1, 1 << 25, 4),
                                     (2, 4, 1, 8), (3, 32, 1, 32)])
def test_selection_of_many_requests_and_tokens(R, W, V, k):
    """The requests' answers do not depend on their place and company; fewer candidates than asked for leave -1.
    (Another number of rows cuts each into other slices, whose sums round otherwise.)"""
    gen = torch.Generator(device="cuda").manual_seed(V)
    x = torch.randn(R * W, V, generator=gen, device="cuda").bfloat16()
    s = torch.randn(R * W, generator=gen, device="cuda")
    got = av.beam_select(x, s, W, k)
    moved = av.beam_select(x.roll(W, 0), s.roll(W), W, k)
    assert all(torch.equal(a.roll(1, 0), b) for a, b in zip(got, moved))
    row = torch.log_softmax(x[:W].double(), -1) + s[:W, None].double()
    n = min(k, W * V)
    # |values| < 64, three roundings to fp32 of at most 2^-19; the sum of 2^25 terms in fp32: at most 2^11 of them
    # one after the other, 2^-13 of it
    assert (got[2][0, :n].double() - row.flatten().topk(n).values).abs().max() < 3 * 2.0 ** -19 + 2.0 ** -13
    assert got[0][0, n:].eq(-1).all() and got[1][0, n:].eq(-1).all() and got[2][0, n:].eq(-float("inf")).all()
    assert av.get_last_device_error()[0] == 0


def test_copies_of_very_many_and_none():
    n = 70000
    cache = torch.arange(2 * n, dtype=torch.int32, device="cuda")[:, None].repeat(1, 4)
    src, dst = torch.arange(n, device="cuda").int(), torch.arange(2 * n - 1, n - 1, -1, device="cuda").int()
    av.copy_states(cache, src, dst)
    assert torch.equal(cache[n:], cache[:n].flip(0))
    # a token each, pages of 16 tokens, one kv head of 8: row r owns page r
    kc, vc = (torch.randint(0, 99, (2 * n, 16, 1, 8), device="cuda").bfloat16() for _ in range(2))
    before = kc.clone(), vc.clone()
    pages = torch.arange(2 * n, dtype=torch.int32, device="cuda")[:, None].contiguous()
    lens = torch.ones(2 * n, dtype=torch.int32, device="cuda")
    av.copy_kvcache(kc, vc, src, dst, pages, lens)
    for a, b in zip((kc, vc), before):
        assert torch.equal(a[n:, 0], b[:n, 0].flip(0)) and torch.equal(a[:, 1:], b[:, 1:]) and torch.equal(a[:n], b[:n])
    assert av.get_last_device_error()[0] == 0


def test_cached_rows_past_32_bits():
    blocks, bs, H, D = 66000, 16, 16, 128                   # 2^15 elements a page: 2.16e9 in all
    kc, vc = (torch.empty(blocks, bs, H, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    kc[blocks - 2:] = torch.randn(2, bs, H, D, device="cuda").bfloat16()
    vc[blocks - 2:] = torch.randn(2, bs, H, D, device="cuda").bfloat16()
    kc[:2], vc[:2] = 0, 0
    pages, lens = i32(blocks - 1, blocks - 2, 1, 0).view(2, 2), i32(20, 20)
    av.copy_kvcache(kc, vc, i32(0), i32(1), pages, lens)
    for x in (kc, vc):
        assert torch.equal(x[1], x[blocks - 1]) and torch.equal(x[0, :4], x[blocks - 2, :4]) and x[0, 4:].eq(0).all()
    assert av.get_last_device_error()[0] == 0


def test_more_candidates_than_beams():
    """Twice as many as beams are chosen, the even ones go on (a caller's own choice among them)."""
    from attention_attn_varlen_gb300.attention import Beams, PagePool
    R, W, V = 3, 4, 1000
    pool = PagePool(R * W * 2, 16, R * W, 2)
    beams = Beams(pool, torch.arange(R * W, dtype=torch.int32, device="cuda").view(R, W))
    gen = torch.Generator(device="cuda").manual_seed(9)
    for _ in range(3):
        x, before, rows = torch.randn(R * W, V, generator=gen, device="cuda"), beams.scores, beams.rows
        tokens, parents, scores = beams.select(x, 2 * W)
        beams.advance(parents[:, ::2], scores[:, ::2])
        assert torch.equal(beams.scores, scores[:, ::2])
        assert torch.equal(beams.rows.sort(1).values, rows.sort(1).values)
        all_ = (before.double()[..., None] + torch.log_softmax(x.double(), -1).view(R, W, V)).flatten(1)
        want = all_.topk(2 * W, 1).values
        # sums of 1,000 terms in fp32, 2^-24 for each addition, and scores below 64 rounded to fp32
        assert ((scores.double() - want).abs() <= 1000 * 2.0 ** -24 + 2.0 ** -18).all()
    assert av.get_last_device_error()[0] == 0
