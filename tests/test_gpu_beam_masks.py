"""beam_select over the whole range of finite logits: masks that are large negative
numbers, rows of nothing else, maxima far above the rest; against the definition in 64 bits.

Which candidates are chosen is exact.  A score is s + (x - log(sum of e^x)) in 64 bits, with the
logarithm as the maximum plus that of an fp32 sum (off by 2^-18 at the very worst, as in the
selection's other tests), rounded to 64 bits on either side, 2^-53 of the maximum each, and
the result to fp32, 2^-24 of it."""
import math

import pytest
import torch

import attention_attn_varlen_gb300 as av

pytestmark = pytest.mark.gpu
INF = float("inf")
MASKS = (-1e9, -1.4e9, -3e9, -5e9, -1e10, -1e12, -1e20, -1e30, -1e36, -1e37, -1e38, -3e38)


def select(logits, scores, W, k):
    N, V = logits.shape
    x = logits.double()
    top = x.max(1, keepdim=True).values
    rest = x - (top + torch.exp(x - top).sum(1, keepdim=True).log())
    want = [], [], []
    for r in range(N // W):
        cand = []
        for b in range(W):
            row = r * W + b
            order = torch.sort(x[row], descending=True, stable=True).indices[:k].tolist()
            s = float(scores[row])
            cand += [(-(s + float(rest[row, t])), b, i, t) for i, t in enumerate(order)]
        cand = sorted(cand)[:k]
        for to, y in zip(want, zip(*((t, b, -m) for m, b, _, t in cand))):
            to.append(list(y))
    return tuple(torch.tensor(y, dtype=t) for y, t in zip(want, (torch.int32, torch.int32, torch.float64)))


def check(logits, W, k, what):
    gen = torch.Generator().manual_seed(len(what))
    scores = -5 * torch.rand(logits.shape[0], generator=gen)
    got = av.beam_select(logits.cuda(), scores.cuda(), W, k)
    want = select(logits, scores, W, k)
    assert av.get_last_device_error()[0] == 0, what
    assert torch.equal(got[0].cpu(), want[0]) and torch.equal(got[1].cpu(), want[1]), what
    err = (got[2].cpu().double() - want[2]).abs()
    top = logits.double().abs().max()
    assert (err <= 2.0 ** -18 + 2.0 ** -24 * want[2].abs() + 2.0 ** -52 * top).all(), (what, err.max())


@pytest.mark.parametrize("R,W,V", [(1, 4, 20000), (3, 2, 2049), (40, 4, 3000), (1, 1, 70001)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_masks_of_large_finite_values(R, W, V, dtype):
    """A few allowed tokens, one in 700, half of them, all but a run at the front, none."""
    gen = torch.Generator().manual_seed(V)
    x = 2 * torch.randn(R * W, V, generator=gen)
    few = torch.zeros(R * W, V, dtype=torch.bool)
    few[:, torch.randint(0, V, (3,), generator=gen)] = True
    some = torch.rand(R * W, V, generator=gen) < 1 / 700
    some[:, -1] = True
    half = torch.rand(R * W, V, generator=gen) < 0.5
    back = torch.arange(V).expand(R * W, V) >= V // 2
    av.get_last_device_error()
    for mask in MASKS:
        for name, allowed in (("few", few), ("some", some), ("half", half), ("back", back), ("none", few & False)):
            check(torch.where(allowed, x, torch.tensor(mask)).to(dtype), W, 8, f"{name} {mask}")
        # one row of the mask alone beside ordinary ones, and another mask in a part of each row
        y = x.clone()
        y[0] = mask
        check(y.to(dtype), W, 8, f"one row {mask}")
        y[:, : V // 3] = 10 * mask if mask > -1e37 else mask / 10
        y[:, V // 3: V // 2] = -1e4
        check(y.to(dtype), W, 8, f"two masks {mask}")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("top", [1e4, 1e6, 1e9, 2e9, 1e10, 1e20, 1e37, 2.3e38, 2.4e38, 3e38])
def test_maxima_of_large_finite_values(dtype, top):
    W, V = 2, 9001
    gen = torch.Generator().manual_seed(3)
    x = 2 * torch.randn(W, V, generator=gen)
    av.get_last_device_error()
    for at in ([4], [4500], [9000], [0, 5000], [1, 2, 3, 8999]):
        y = x.clone()
        y[:, at] = top
        check(y.to(dtype), W, 8, f"at {at}")
        y[0, ::7] = -top                                     # both ends of the range in a row
        check(y.to(dtype), W, 8, f"both {at}")
    check(torch.full((W, V), top).to(dtype), W, 8, "all")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_logits_of_every_size(dtype):
    """Signs and magnitudes spread over the type's whole range."""
    W, V = 3, 12007
    gen = torch.Generator().manual_seed(8)
    av.get_last_device_error()
    for low, high in ((-3.0, 38.4), (8.0, 11.0), (0.0, 9.3), (36.0, 38.4)):
        size = 10.0 ** (low + (high - low) * torch.rand(W, V, generator=gen, dtype=torch.float64))
        for sign in (torch.where(torch.rand(W, V, generator=gen) < 0.5, -1.0, 1.0), torch.full((W, V), -1.0)):
            check((sign.double() * size).float().to(dtype), W, 16, f"{low} {high}")
    assert math.isfinite(float(torch.tensor(10.0 ** 38.4).to(dtype)))
