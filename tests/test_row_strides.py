"""Rows that lie on one another (a tensor expanded along its rows has row stride 0,
which the library reads as packed) are refused before anything is launched."""
import pytest
import torch

import attention_attn_varlen_gb300 as av


def _expanded(n, heads, dim, device="cpu"):
    return torch.zeros(1, heads, dim, dtype=torch.bfloat16, device=device).expand(n, heads, dim)


@pytest.mark.parametrize("rows_of", [lambda t: av._rows(t, "k", 2, 64), lambda t: av._tokens(t, "k", -1, len(t), 2, 64)])
def test_row_strides(rows_of):
    assert rows_of(torch.zeros(5, 2, 64, dtype=torch.bfloat16)) == 128
    assert rows_of(torch.zeros(5, 6, 64, dtype=torch.bfloat16)[:, 2:4]) == 384
    assert rows_of(_expanded(1, 2, 64)) == 128           # one row: its stride is not used
    assert rows_of(torch.zeros(0, 2, 64, dtype=torch.bfloat16)) == 128
    with pytest.raises(ValueError, match="overlap"):
        rows_of(_expanded(5, 2, 64))
    with pytest.raises(ValueError, match="overlap"):
        rows_of(torch.zeros(1000, dtype=torch.bfloat16).as_strided((5, 2, 64), (64, 64, 1)))


@pytest.mark.gpu
def test_every_entry_that_takes_rows_refuses_them():
    H, D, n = 2, 64, 5
    x, flat = torch.zeros(n, H, D, dtype=torch.bfloat16, device="cuda"), _expanded(n, H, D, "cuda")
    cache = torch.zeros(4, 16, H, D, dtype=torch.bfloat16, device="cuda")
    i32 = lambda *y: torch.tensor(y, dtype=torch.int32, device="cuda")  # noqa: E731
    slots, cu, one = torch.arange(n, device="cuda"), i32(0, n), i32(*[1] * n)
    table = torch.zeros(n, 1, dtype=torch.int32, device="cuda")
    pos, inv, g = torch.arange(n, dtype=torch.int32, device="cuda"), torch.ones(D // 2, device="cuda"), torch.zeros(H, device="cuda")
    states, ids = torch.zeros(n, H, D, D, device="cuda"), torch.arange(n, dtype=torch.int32, device="cuda")
    calls = [lambda *t: av.store_kvcache(*t[1:], cache, cache.clone(), slots),
             lambda *t: av.attn_varlen_fwd(*t, cu, cu, n, n),
             lambda *t: av.rope_store_kvcache(*t, pos, inv, cache, cache.clone(), slots),
             lambda *t: av.linear_attn_varlen_fwd(*t, g, cu, n),
             lambda *t: av.linear_attn_decode(*t, g, states, ids)]
    for call in calls:
        call(x, x, x)
        for bad in ((flat, x, x), (x, flat, x), (x, x, flat)):
            if call is calls[0] and bad[0] is flat:
                continue                                 # the store takes no q
            with pytest.raises(ValueError, match="overlap"):
                call(*bad)
    av.attn_decode_paged(x, cache, cache, one, table)
    with pytest.raises(ValueError, match="overlap"):
        av.attn_decode_paged(flat, cache, cache, one, table)
    for out in (flat, torch.zeros(1000, dtype=torch.bfloat16, device="cuda").as_strided((n, H, D), (D, D, 1))):
        with pytest.raises(ValueError, match="overlap"):
            av.attn_varlen_fwd(x, x, x, cu, cu, n, n, out=out)
        with pytest.raises(ValueError, match="overlap"):
            av.rope_store_kvcache(x, x, None, pos, inv, q_out=out)
        with pytest.raises(ValueError, match="overlap"):
            av.linear_attn_varlen_fwd(x, x, x, g, cu, n, out=out)
    m = torch.zeros(1, 40, device="cuda")
    av.softmax_rows(m.expand(1, 40))
    with pytest.raises(ValueError, match="overlap"):
        av.softmax_rows(m.expand(8, 40))
    with pytest.raises(ValueError, match="overlap"):
        av.softmax_rows(torch.zeros(8, 40, device="cuda"), out=m.expand(8, 40))
    torch.cuda.synchronize()
    assert av.get_last_device_error()[0] == 0
