"""beam_select, beam_rows, copy_states and copy_kvcache on the GPU against plain Python.

Which candidates are chosen is exact.  A score is the 64-bit one rounded to fp32 (2^-24
of it), with the logarithm of a sum of exponentials in fp32: each exponential is off by
2^-21 at most (its argument's rounding and the function's), sums of a lane's up to 64
batches of 32 terms, eight warps and 64 slices by 2^-18 at the very worst, as is the logarithm."""
import pytest
import torch

import attention_attn_varlen_gb300 as av
from _delta_reference import beam_rows, select

pytestmark = pytest.mark.gpu
INF = float("inf")


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def check(logits, scores, W, k, what=""):
    got = av.beam_select(logits.cuda(), scores.cuda(), W, k)
    want = select(logits, scores, W, k)
    assert torch.equal(got[0].cpu(), want[0]) and torch.equal(got[1].cpu(), want[1]), what
    some = torch.isfinite(want[2])
    assert torch.equal(torch.isfinite(got[2].cpu()), some)
    err = (got[2].cpu().double() - want[2])[some].abs()
    assert (err <= 2.0 ** -18 + 2.0 ** -24 * want[2][some].abs()).all(), what
    return got


@pytest.mark.parametrize("R,W,V,k", [(1, 1, 1, 1), (1, 1, 7, 3), (3, 4, 100, 8), (2, 8, 2047, 16), (1, 4, 2048, 4),
                                     (5, 3, 2049, 6), (2, 32, 5000, 32), (1, 2, 70001, 32), (40, 5, 8193, 10),
                                     (1, 1, 200000, 2), (300, 4, 999, 8)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_selection(R, W, V, k, dtype):
    gen = torch.Generator().manual_seed(R + V)
    logits = (2 * torch.randn(R * W, V, generator=gen)).to(dtype)
    scores = -5 * torch.rand(R * W, generator=gen)
    av.get_last_device_error()
    check(logits, scores, W, k)
    # a part of the vocabulary and some beams ruled out
    logits[torch.rand(R * W, V, generator=gen) < 0.6] = -INF
    scores[torch.rand(R * W, generator=gen) < 0.3] = -INF
    check(logits, scores, W, k, "masked")
    assert av.get_last_device_error()[0] == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_equal_and_extreme_logits(dtype):
    """Ties go to the lowest beam and token, wherever they lie; sorted rows; masks of the
    type's lowest value; both zeros are one value."""
    W, V, k = 2, 9000, 16
    low = torch.finfo(dtype).min
    flat = torch.zeros(W, V, dtype=dtype)
    rising = torch.linspace(-8, 8, V).to(dtype).expand(W, V)
    falling = rising.flip(1)
    few = torch.full((W, V), -3.0, dtype=dtype)
    few[0, 8990:] = 2.0
    few[1, ::1000] = 2.0
    lowest = torch.full((W, V), low, dtype=dtype)
    mixed = lowest.clone()
    mixed[:, 77::500] = 1.5
    zeros = flat.clone()
    zeros[:, ::2] = -0.0
    same = (torch.randn(1, V, generator=torch.Generator().manual_seed(1)) * 3).to(dtype).expand(W, V).contiguous()
    for name, x in dict(flat=flat, rising=rising, falling=falling, few=few, lowest=lowest, mixed=mixed, zeros=zeros,
                        same=same).items():
        check(x.contiguous(), torch.zeros(W), W, k, name)
        check(x.contiguous(), torch.tensor([-INF, 0.0]), W, k, name)
    # fewer candidates than asked for, and none
    none = torch.full((W, V), -INF, dtype=dtype)
    none[1, 5000] = 1.0
    check(none, torch.zeros(W), W, k, "one")
    none[1, 5000] = -INF
    check(none, torch.zeros(W), W, k, "none")
    assert av.get_last_device_error()[0] == 0


def test_strides_and_mistaken_values():
    gen = torch.Generator().manual_seed(4)
    W, V, k = 3, 4097, 6
    for dtype in (torch.bfloat16, torch.float32):
        wide = (2 * torch.randn(2 * W, V + 31, generator=gen)).to(dtype)
        dev = wide.cuda()
        scores = -torch.rand(2 * W, generator=gen)
        for at in (0, 1, 8):
            x = dev[:, at:at + V]
            got = av.beam_select(x, scores.cuda(), W, k)
            want = select(wide[:, at:at + V], scores, W, k)
            assert torch.equal(got[0].cpu(), want[0]) and torch.equal(got[1].cpu(), want[1])
        # identical rows at any alignment give identical sums: the lowest beam comes first
        odd = wide[:1, :V].expand(2 * W, V).contiguous()
        check(odd, torch.zeros(2 * W), W, k, "same")
        av.get_last_device_error()
        # a NaN or +inf takes its beam's candidates away, and is reported
        for bad in (float("nan"), INF):
            x = wide[:, :V].clone()
            x[1, 4000] = bad
            got = av.beam_select(x.cuda(), scores.cuda(), W, k)
            assert av.get_last_device_error()[0] == 8
            assert not got[1][0].eq(1).any()
            s = scores.clone()
            s[1] = -INF
            x[1] = 0
            assert torch.equal(got[0].cpu(), select(x, s, W, k)[0])
            s[1] = bad
            got = av.beam_select(x.cuda(), s.cuda(), W, k)
            assert av.get_last_device_error()[0] == 8
            assert not got[1][0].eq(1).any()


def test_captured_and_shared_workspace():
    gen = torch.Generator().manual_seed(6)
    sizes = [(4, 4, 30000, 8), (1, 8, 5001, 16)]
    ws = torch.empty(max(av.beam_select_workspace_size(R, W, V, k) for R, W, V, k in sizes), dtype=torch.uint8,
                     device="cuda")
    runs = []
    for R, W, V, k in sizes:
        x = torch.randn(R * W, V, generator=gen).cuda()
        s = torch.zeros(R * W, device="cuda")
        want = av.beam_select(x, s, W, k)
        out = tuple(torch.empty_like(y) for y in want)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            av.beam_select(x, s, W, k, out=out, workspace=ws)
        runs.append((graph, want, out, x, s))
    for _ in range(3):
        for graph, *_ in runs:
            graph.replay()
    torch.cuda.synchronize()
    for _, want, out, *_ in runs:
        assert all(torch.equal(a, b) for a, b in zip(want, out))


@pytest.mark.parametrize("R,W", [(1, 1), (1, 2), (3, 4), (9, 5), (70, 16), (5, 32)])
def test_rows_of_the_next_beams(R, W):
    gen = torch.Generator().manual_seed(R * W)
    rows = torch.randperm(R * W + 7, generator=gen)[:R * W].to(torch.int32).view(R, W)
    av.get_last_device_error()
    for parents in (torch.randint(0, W, (R, W), generator=gen), torch.zeros(R, W), torch.full((R, W), W - 1),
                    torch.arange(W).flip(0).expand(R, W), torch.randint(-1, W, (R, W), generator=gen),
                    torch.full((R, W), -1)):
        parents = parents.to(torch.int32).contiguous()
        want = beam_rows(parents, rows)
        got = av.beam_rows(parents.cuda(), rows.cuda())
        assert torch.equal(got[0].cpu(), want[0]) and torch.equal(got[1].cpu(), want[1])
        into = rows.cuda()                                   # in place
        av.beam_rows(parents.cuda(), into, out=(into, torch.empty_like(into)))
        assert torch.equal(into.cpu(), want[0])
    assert av.get_last_device_error()[0] == 0
    parents[0, 0] = W
    got = av.beam_rows(parents.cuda(), rows.cuda())
    assert av.get_last_device_error()[0] == 6
    assert torch.equal(got[0].cpu(), beam_rows(parents, rows)[0])


@pytest.mark.parametrize("shape,dtype", [((9, 4, 64, 64), torch.float32), ((9, 3, 5, 8), torch.bfloat16),
                                         ((9, 16), torch.uint8), ((9, 2, 128, 128), torch.float32),
                                         ((9, 100, 1001, 4), torch.float32)])
def test_copies_of_states(shape, dtype):
    gen = torch.Generator().manual_seed(len(shape))
    cache = torch.randint(0, 100, shape, generator=gen).to(dtype)
    src, dst = [3, -1, 3, 7, 5, -1], [0, 2, 8, 1, 5, 4]
    dev = cache.cuda()
    av.get_last_device_error()
    av.copy_states(dev, i32(src), i32(dst))
    want = cache.clone()
    for a, b in zip(src, dst):
        if a >= 0:
            want[b] = cache[a]
    assert torch.equal(dev.cpu(), want) and av.get_last_device_error()[0] == 0
    for a, b in ((9, 1), (1, 9), (1, -1)):                   # out of range: skipped
        av.copy_states(dev, i32([a, 3]), i32([b, 2]))
        assert av.get_last_device_error()[0] == 6
        want[2] = want[3]
        assert torch.equal(dev.cpu(), want)
    av.copy_states(dev, i32([]), i32([]))
    assert torch.equal(dev.cpu(), want)


@pytest.mark.parametrize("Hkv,D,bs,v16", [(2, 64, 16, True), (8, 128, 64, False), (1, 66, 16, True), (1, 64, 256, True)])
@pytest.mark.parametrize("first", [False, True])
def test_copies_of_cached_rows(Hkv, D, bs, v16, first):
    gen = torch.Generator().manual_seed(D + bs)
    rows, M = 6, 5
    lens = torch.tensor([3 * bs + 5, 2 * bs, 3 * bs + 5, 0, 2 * bs, 3 * bs + 5], dtype=torch.int32)
    pages = torch.randperm(rows * M + 3, generator=gen)[:rows * M].view(rows, M).to(torch.int32)
    for r in range(rows):
        pages[r, -(-int(lens[r]) // bs):] = -1
    firsts = torch.tensor([bs + 3, 5, bs + 3, 0, 2 * bs, 4 * bs], dtype=torch.int32)
    make = lambda dt: torch.randint(0, 100, (rows * M + 3, bs, Hkv, D), generator=gen).to(dt)  # noqa: E731
    caches = [make(torch.bfloat16), make(torch.bfloat16)] + ([make(torch.float16)] if v16 else [])
    src, dst = [0, 4, -1, 3, 1], [2, 1, 0, 3, 1]
    src, dst = src[:4], dst[:4]

    def copied(xs, pairs):
        out = [x.clone() for x in xs]
        for a, b in pairs:
            for t in range(int(firsts[a]) if first else 0, int(lens[a])):
                for x, y in zip(xs, out):
                    y[pages[b, t // bs], t % bs] = x[pages[a, t // bs], t % bs]
        return out

    dev = [x.cuda() for x in caches]
    args = (pages.cuda(), lens.cuda())
    kw = dict(first_tokens=firsts.cuda() if first else None, v16_cache=dev[2] if v16 else None)
    av.get_last_device_error()
    av.copy_kvcache(dev[0], dev[1], i32(src), i32(dst), *args, **kw)
    assert av.get_last_device_error()[0] == 0
    want = copied(caches, [(a, b) for a, b in zip(src, dst) if a >= 0 and a != b])
    assert all(torch.equal(x.cpu(), y) for x, y in zip(dev, want))
    # rows of other lengths or out of range are skipped, and so are tokens whose page is missing
    for a, b in ((0, 1), (6, 0), (0, 6), (0, -1)):
        av.copy_kvcache(dev[0], dev[1], i32([a]), i32([b]), *args, **kw)
        assert av.get_last_device_error()[0] == 6
        assert all(torch.equal(x.cpu(), y) for x, y in zip(dev, want))
    hole = pages.clone()
    hole[5, 2] = rows * M + 3
    av.copy_kvcache(dev[0], dev[1], i32([0]), i32([5]), hole.cuda(), lens.cuda(), **kw)
    assert av.get_last_device_error()[0] == 6
    for t in range(int(firsts[0]) if first else 0, int(lens[0])):
        for x, y in zip(want, dev):
            if t // bs != 2:
                x[pages[5, t // bs], t % bs] = x[pages[0, t // bs], t % bs]
    assert all(torch.equal(x.cpu(), y) for x, y in zip(dev, want))
