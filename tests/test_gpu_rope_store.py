"""rope_store_kvcache on the GPU against the definition in 64 bits.

Tolerance.  The rotated element u = s (a cos - b sin) is rounded once to bf16:
at most 2^-8 of it.  Before that, fp32: the sine and cosine are off by at most
2^-23 (angle: 2^-24 of half a turn rounding to fp32, times pi, plus the
function's own error), three roundings of 2^-24, each of terms of size s (|a| +
|b|): together below 2^-20 s (|a| + |b|).  The value rounded may move to the
next bf16 boundary by that, which the sum covers.
"""
import numpy as np
import pytest
import torch

import attention_attn_varlen_gb300 as av
from _step_reference import rope

pytestmark = pytest.mark.gpu


def _close(got, ref, size, what):
    err = (got.double().cpu() - ref).abs()
    tol = 2.0 ** -8 * ref.abs() + 2.0 ** -20 * size
    assert torch.isfinite(got.float()).all(), what
    assert (err <= tol).all(), f"{what}: {(err - tol).max():.3e}"


def _size(x, half, inter, scale):
    """s (|a| + |b|) of the pair an element belongs to; 0 where it is copied."""
    y = torch.zeros_like(x, dtype=torch.float64)
    a = x.double().abs()
    if inter:
        m = a[..., 0:2 * half:2] + a[..., 1:2 * half:2]
        y[..., 0:2 * half:2] = y[..., 1:2 * half:2] = m
    else:
        m = a[..., :half] + a[..., half:2 * half]
        y[..., :half] = y[..., half:2 * half] = m
    return scale * y


def _inv(half, base=10000.0):
    return (base ** (-torch.arange(half, dtype=torch.float64) / half)).float()


@pytest.mark.parametrize("N,Hq,Hkv,D,rot,axes,inter,scale,packed,v16", [
    (1, 1, 1, 64, 64, 1, False, 1.0, True, False),
    (5, 8, 2, 128, 128, 1, False, 1.0, False, True),
    (64, 32, 8, 128, 128, 3, False, 1.0, False, False),
    (1237, 16, 16, 64, 32, 1, True, 1.3, False, True),
    (333, 6, 2, 128, 64, 4, True, 0.7, True, False),
    (700, 10, 2, 128, 128, 3, True, 1.0, False, False),
    (9, 3, 1, 80, 40, 2, False, 1.0, False, True),          # a rotated half of 20: one element at a time
    (17, 5, 5, 6, 4, 1, True, 1.0, True, True),
    (21, 2, 1, 256, 256, 1, False, 1.0, False, False),
    (40, 4, 2, 96, 96, 1, False, 1.0, False, True)])
def test_rotates_and_stores(N, Hq, Hkv, D, rot, axes, inter, scale, packed, v16):
    gen = torch.Generator().manual_seed(N + D)
    rng = np.random.default_rng(N + D)
    half = rot // 2
    qkv = (torch.randn(N, Hq + 2 * Hkv, D, generator=gen) * 3).to(torch.bfloat16)
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    dev = qkv.cuda()
    qd, kd, vd = dev[:, :Hq], dev[:, Hq:Hq + Hkv], dev[:, Hq + Hkv:]
    if packed:
        qd, kd, vd = qd.contiguous(), kd.contiguous(), vd.contiguous()
    pos = torch.from_numpy(rng.integers(0, 1 << 20, size=(axes, N)).astype(np.int32))
    axis = None if axes == 1 else [int(x) for x in rng.integers(0, axes, size=half)]
    inv = _inv(half)
    slots = rng.permutation(2 * N + 5)[:N].astype(np.int64)
    slots[::7] = -1
    slots_d = torch.from_numpy(slots).cuda()
    sentinel = torch.from_numpy(rng.integers(0, 1 << 14, size=(2 * N + 5, Hkv, D)).astype(np.int16))
    kc, vc = sentinel.view(torch.bfloat16).cuda(), sentinel.view(torch.bfloat16).cuda()
    vh = sentinel.view(torch.float16).cuda() if v16 else None
    av.get_last_device_error()
    pd = pos.cuda() if axes > 1 else pos[0].cuda()
    got, k_out = av.rope_store_kvcache(qd, kd, vd, pd, inv.cuda(), kc, vc, slots_d, pair_axis=axis, interleaved=inter,
                                       scale=scale, v16_cache=vh, return_k=True)
    torch.cuda.synchronize()
    assert av.get_last_device_error()[0] == 0
    rq, rk = rope(q, pos, inv, axis, inter, scale), rope(k, pos, inv, axis, inter, scale)
    _close(got, rq, _size(q, half, inter, scale), "q")
    _close(k_out, rk, _size(k, half, inter, scale), "k")
    # elements past the rotated part are copied bit for bit
    assert torch.equal(got.cpu()[..., rot:], q[..., rot:])
    # the caches hold the rotated k, v and V / 16 at the slots, and nothing else changed
    keep = torch.from_numpy(slots >= 0)
    at = torch.from_numpy(slots[slots >= 0])
    ek, ev = sentinel.clone(), sentinel.clone()
    ek[at] = k_out.cpu()[keep].view(torch.int16)
    ev[at] = v.contiguous()[keep].view(torch.int16)
    assert torch.equal(kc.cpu().view(torch.int16), ek)
    assert torch.equal(vc.cpu().view(torch.int16), ev)
    if v16:
        eh = sentinel.clone()
        eh[at] = (v.contiguous()[keep].float() / 16).half().view(torch.int16)
        assert torch.equal(vh.cpu().view(torch.int16), eh)


@pytest.mark.parametrize("D,inter", [(128, False), (128, True), (10, False)])
def test_in_place_and_without_a_cache(D, inter):
    gen = torch.Generator().manual_seed(D)
    q = torch.randn(37, 3, D, generator=gen).to(torch.bfloat16)
    k = torch.randn(37, 1, D, generator=gen).to(torch.bfloat16)
    pos = torch.arange(37, dtype=torch.int32) * 1000 - 9000          # negative ones too
    inv = _inv(D // 2)
    qd, kd = q.cuda(), k.cuda()
    a, b = av.rope_store_kvcache(qd, kd, None, pos.cuda(), inv.cuda(), interleaved=inter)
    qi, ki = av.rope_store_kvcache(qd, kd, None, pos.cuda(), inv.cuda(), interleaved=inter, q_out=qd, k_out=kd,
                                   return_k=True)
    assert qi is qd and ki is kd and torch.equal(qd, a) and torch.equal(kd, b)
    _close(a, rope(q, pos, inv, None, inter, 1.0), _size(q, D // 2, inter, 1.0), "q")
    _close(b, rope(k, pos, inv, None, inter, 1.0), _size(k, D // 2, inter, 1.0), "k")


def test_far_positions_keep_their_fraction_of_a_turn():
    """Positions up to 2^31 - 1: the angle of the fastest pair is still right to
    2^-24 of a turn (inv_freq / 2 pi carries 53 bits)."""
    pos = torch.tensor([0, 1, 2 ** 20 + 1, 10 ** 6, 2 ** 24 + 1, 2 ** 31 - 1, -2 ** 31], dtype=torch.int32)
    D = 64
    inv = _inv(32, 500000.0)
    q = torch.ones(len(pos), 1, D, dtype=torch.bfloat16)
    got, _ = av.rope_store_kvcache(q.cuda(), q.cuda(), None, pos.cuda(), inv.cuda())
    # integer arithmetic on the exact binary value of inv_freq / 2 pi, to 200 bits
    from fractions import Fraction
    two_pi = 2 * Fraction(314159265358979323846264338327950288419716939937510582097494459230781640628620899, 10 ** 80)
    ref = torch.zeros(len(pos), 1, D, dtype=torch.float64)
    for t, p in enumerate(pos.tolist()):
        for i in range(32):
            turn = Fraction(p) * Fraction(float(inv[i])) / two_pi
            ang = float((turn - (turn.numerator // turn.denominator)) * two_pi)
            ref[t, 0, i] = np.cos(ang) - np.sin(ang)
            ref[t, 0, 32 + i] = np.sin(ang) + np.cos(ang)
    err = (got.double().cpu() - ref).abs()
    assert (err <= 2.0 ** -8 * ref.abs() + 2.0 ** -19).all(), err.max()


def test_a_bad_slot_is_flagged_and_not_written():
    q = torch.ones(4, 2, 64, dtype=torch.bfloat16, device="cuda")
    kc = torch.zeros(16, 2, 64, dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    av.get_last_device_error()
    slots = torch.tensor([0, 99, -1, 3], dtype=torch.int64, device="cuda")
    pos = torch.zeros(4, dtype=torch.int32, device="cuda")
    av.rope_store_kvcache(q, q, q, pos, _inv(32).cuda(), kc, vc, slots)
    st, word = av.get_last_device_error()
    assert st == 6 and word & 1
    assert kc[0].eq(1).all() and kc[3].eq(1).all() and kc[1].eq(0).all() and vc[2].eq(0).all()
    v = q.clone()
    v[3, 1, 5] = 3.0e6
    v16 = torch.zeros(16, 2, 64, dtype=torch.float16, device="cuda")
    av.rope_store_kvcache(q, q, v, pos, _inv(32).cuda(), kc, vc,
                          torch.tensor([0, 1, -1, 3], dtype=torch.int64, device="cuda"), v16_cache=v16)
    st, word = av.get_last_device_error()
    assert st == 8 and word & 4 and v16[3, 1, 5].item() == 65504.0


def test_no_tokens():
    q = torch.empty(0, 2, 64, dtype=torch.bfloat16, device="cuda")
    a, b = av.rope_store_kvcache(q, q, None, torch.empty(0, dtype=torch.int32, device="cuda"), _inv(32).cuda())
    assert a.shape == q.shape and b.shape == q.shape


def test_slots_and_rows_past_32_bits_of_offset():
    """A slot further than 2^31 elements into the caches, rows of q as far apart."""
    N, H, D, num = 3, 2, 128, (1 << 23) + 7                # 2^8 elements a slot
    gen = torch.Generator().manual_seed(6)
    q, k, v = (torch.randn(N, H, D, generator=gen).to(torch.bfloat16) for _ in range(3))
    stride = 1 << 30
    qd = torch.empty((N - 1) * stride + H * D, dtype=torch.bfloat16, device="cuda").as_strided((N, H, D), (stride, D, 1))
    qd.copy_(q.cuda())
    kc, vc = (torch.empty(num, H, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    pos = torch.tensor([0, 7, 2 ** 31 - 1], dtype=torch.int32)
    slots = torch.tensor([num - 1, 5, num - 6])
    inv = _inv(D // 2)
    got, kr = av.rope_store_kvcache(qd, k.cuda(), v.cuda(), pos.cuda(), inv.cuda(), kc, vc, slots.cuda(), return_k=True)
    _close(got, rope(q, pos, inv, None, False, 1.0), _size(q, D // 2, False, 1.0), "q")
    assert torch.equal(kc[slots.cuda()], kr) and torch.equal(vc[slots.cuda()].cpu(), v)
    assert av.get_last_device_error()[0] == 0
